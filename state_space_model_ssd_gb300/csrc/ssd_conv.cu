// Short causal depthwise convolution over the tokens of packed or dense sequences, with its
// carried window, and its backward pass.  Channel c, K taps, sequence tokens i = 0, 1, ...
// at positions p0 + i:
//
//   pre[i] = b + sum_{j < K} w[c][K-1-j] u[i-j],   u[-m]: the carried state's token at p0 - m
//   out[i] = pre[i] sigmoid(pre[i])                (or pre[i])
//
//   g[i]   = dout[i] s (1 + pre (1 - s)),  s = sigmoid(pre[i])
//   du[i]  = sum_{j < K} w[K-1-j] g[i+j]   (tokens of the same sequence)
//   dw[k]  = sum_i g[i] u[i-(K-1-k)],  db = sum_i g[i]
//
// The state of a sequence is K rows of channels; row p mod K holds the token at position p.
// A step at position p reads the rows of p-1 .. p-K+1 and writes only row p mod K, which no
// reader of that step needs: the one-token kernel needs no second buffer and no barrier
// between blocks.
//
// Both passes are bound by HBM (forward: u in, out out; backward: u, dout in, du out).  A lane
// owns VEC neighbouring channels and its warp walks a run of tokens with the window in
// registers, so every element is loaded once, plus K-1 tokens at the run's start (forward) or
// 2 (K-1) around it (backward, which recomputes g there) that its neighbours have brought into
// L2.  Rows that all start on 16 bytes come as tiles of eight tokens, which one lane has copied by
// TMA (in the backward's arithmetic, 25 instructions an element, four separate copies by four
// lanes cost nine more: such a copy takes its operands from uniform registers, lane by lane).
// Groups without an end of a sequence or of the run in reach take a path without any checks.
//
// GB300, bf16, K = 4, SiLU: forward of 32768 x 5376 119 us (88 % of the measured copy rate on 2
// bytes in and 2 out an element), of 65536 packed tokens x 1792 91 us (76 %: the B and C pieces
// fill half of their blocks' lanes); backward of 32768 x 5376 219 us (71 % on 6 bytes an
// element, its partial sums included), of 65536 packed tokens x 1792 157 us (66 %).  The backward
// fills neither memory nor the issue slots (at half the size DRAM 58 %, SM 48 % busy): sixteen warps
// an SM, of 128 registers a thread, wait for the chain of a token's taps, sigmoid, slope and sums
// (25 instructions an element).  Four channels a lane measured best: two 342 us for their overhead,
// eight 295 us for want of warps.  Float32, 32768 x 5376: forward 244, backward 368 us (85 % both).
// Rows off 16 bytes (pairs or single elements): forward 43 to 68 %, backward 20 to 53 %.
#include <limits.h>

#include "layer_device.cuh"
#include "layer_host.cuh"
#include "layer_team.cuh"
#include "tc_common.cuh"

namespace ssd {
namespace layer {

namespace {

constexpr int kLanes = 32;   // channel vectors a block covers
constexpr int kRuns = 8;     // runs of tokens a block covers

struct ConvArgs {
    const void* u;
    const void* w;
    const void* b;
    const int* cu;
    const int* pos;
    const void* init;
    void* out[3];         // forward outputs, or the backward's dout (read only)
    const void* dfinal;
    void* final_state;
    void* du;
    void* dinit;
    float* partial;
    long long T, L;       // all tokens, tokens per dense row
    long long us, dus;    // token strides of u and du, elements
    long long C;
    int off1, off2;       // first channel of pieces 1 and 2
    int blk1, blk2;       // and their first blocks of channels
    int width[3];
    int nseq;             // sequences (dense rows or packed)
    int run;              // tokens a thread walks
    int nrunblk;          // blocks along the tokens
    int nchblk;           // blocks along the channels
    int wbf16;
    int* status;
};

// Tiles of the tensors that a kernel reads: u, and in the backward the pieces of dout.
struct ConvMaps {
    CUtensorMap u, dout[3];
};

struct Seq {
    int s;
    long long start, end;
    bool live;            // false: tokens after the last packed sequence
};

__device__ __forceinline__ long long clampll(long long v, long long lo, long long hi) {
    return v < lo ? lo : v > hi ? hi : v;
}

// The sequence of token t.  Packed: the first s whose end lies beyond t; start and end are
// clamped around t, so that a malformed cu_seqlens gives wrong values, never an access out
// of range.  Tokens from cu[nseq] on belong to no sequence.
__device__ __forceinline__ Seq seq_of(const ConvArgs& a, long long t) {
    Seq q;
    q.live = true;
    if (!a.cu) {
        q.s = (int)(t / a.L);
        q.start = q.s * a.L;
        q.end = q.start + a.L;
        return q;
    }
    int lo = 0, hi = a.nseq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    q.s = lo;
    q.start = lo == 0 ? 0 : clampll(a.cu[lo], 0, t);
    q.live = lo < a.nseq;
    q.end = q.live ? clampll(a.cu[lo + 1], t + 1, a.T) : a.T;
    return q;
}
// Sequence s as a whole (possibly empty).
__device__ __forceinline__ Seq seq_at(const ConvArgs& a, int s) {
    Seq q;
    q.s = s;
    q.live = true;
    if (!a.cu) {
        q.start = s * a.L;
        q.end = q.start + a.L;
    } else {
        q.start = s == 0 ? 0 : clampll(a.cu[s], 0, a.T);
        q.end = clampll(a.cu[s + 1], q.start, a.T);
    }
    return q;
}

// An offset from a run's first token, where it lies in reach of the run.
__device__ __forceinline__ int near(long long v) { return (int)clampll(v, -(1 << 29), 1 << 29); }

template <int K>
__device__ __forceinline__ int state_row(long long p) {
    const int r = (int)(p % K);
    return r < 0 ? r + K : r;
}

// Token i of the sequence that starts at q.start (i < 0: from the carried state), channels
// c .. c + VEC.
template <typename T, int VEC, int K>
__device__ __forceinline__ void token(const ConvArgs& a, const Seq& q, long long i, long long c,
                                      float* f) {
    Pack<T, VEC> v;
    if (i >= 0) {
        v.load(static_cast<const T*>(a.u) + (q.start + i) * a.us + c);
    } else if (a.init && q.live) {
        const long long p0 = a.pos ? a.pos[q.s] : 0;
        v.load(static_cast<const T*>(a.init) + ((long long)q.s * K + state_row<K>(p0 + i)) * a.C + c);
    } else {
        v.zero();
    }
    v.get(f);
}

// Weights and bias of a block's channels, transposed to [K + 1][channels] in shared memory
// (row K is the bias): a thread's VEC channels are then neighbours in every row.
template <int VEC, int K>
__device__ __forceinline__ void stage_weights(const ConvArgs& a, long long c0, int n,
                                              float (*ws)[kLanes * VEC]) {
    const int tid = threadIdx.y * kLanes + threadIdx.x;
    for (int i = tid; i < n * K; i += kLanes * kRuns)
        ws[i % K][i / K] = param(a.w, c0 * K + i, a.wbf16);
    for (int i = tid; i < n; i += kLanes * kRuns) ws[K][i] = a.b ? param(a.b, c0 + i, a.wbf16) : 0.f;
    __syncthreads();
}

// The tokens of a warp's run on their way to it, in groups of kGroup: as tiles of the block's
// channels that one lane has copied (TMA) into a ring of kGroups groups in shared memory, or, in
// vectors of less than 16 bytes, through registers one group ahead.  N tensors.
// Two groups of eight tokens (three measured 2 to 5 % slower); where a token of both tensors takes
// 1 KB (float32 backward), three groups of four tokens, for two blocks an SM.
constexpr int group_of(int vec, int esize, int n) { return vec * esize * n > 16 ? 4 : 8; }
constexpr int groups_of(int vec, int esize, int n) { return vec * esize * n > 16 ? 3 : 2; }
struct RunBars {
    uint64_t full[kRuns][3];
};
template <typename T, int VEC, int N>
struct Run {
    static constexpr bool BULK = VEC >= 4;
    static constexpr int kGroup = group_of(VEC, sizeof(T), N), kGroups = groups_of(VEC, sizeof(T), N);
    static constexpr int line = kLanes * VEC * (int)sizeof(T);  // a token of a tensor in the ring
    static constexpr int tile = kGroup * line;
    Pack<T, VEC> next[BULK ? 1 : kGroup][N];
    const T* src[N];  // the next token to load, this lane's channels
    long long stride[N];
    const CUtensorMap* map[N];
    int col[N];       // the block's first channel in each map
    int token;        // the next to load
    int left;         // groups (single loads: tokens) still to load (groups as wait_copy has it)
    char* ring;       // this warp's
    uint64_t* full;
    int fill, stage;
    uint32_t parity;
    int* status;

    // `tokens` (perhaps none) from t0 on; every lane of the warp calls it.
    __device__ __forceinline__ void begin(long long t0, int tokens, char* all, RunBars* bars,
                                          int* status_word) {
        left = BULK ? (tokens + kGroup - 1) / kGroup : tokens;
        if constexpr (BULK) {
            token = (int)t0;
            ring = all + threadIdx.y * (kGroups * N * tile);
            full = bars->full[threadIdx.y];
            fill = stage = 0;
            parity = 0;
            status = status_word;
            if (threadIdx.x == 0) {
                for (int s = 0; s < kGroups; ++s) tc::mbar_init(&full[s], 1);
                tc::fence_mbar_init();
            }
            __syncwarp();
        }
    }
    // tensor k: its map and the block's first channel there, or token t0 at that channel
    template <int K>
    __device__ __forceinline__ void tensor(const CUtensorMap* m, int c, const T* p, long long by) {
        if constexpr (BULK) {
            map[K] = m;
            col[K] = c;
        } else {
            src[K] = p + threadIdx.x * VEC;
            stride[K] = by;
        }
    }
    __device__ __forceinline__ void start() {
        if constexpr (BULK) {
#pragma unroll
            for (int s = 0; s < kGroups; ++s) issue();
        } else {
            fetch();
        }
    }
    // Tiles are whole: tokens beyond the last are zeros, or a neighbour's that is not looked at.
    __device__ __forceinline__ void issue() {
        if (left <= 0) return;
        if (threadIdx.x == 0) {
            tc::mbar_expect_tx(&full[fill], N * tile);
#pragma unroll
            for (int k = 0; k < N; ++k)
                tc::tma_load_2d(ring + (fill * N + k) * tile, map[k], &full[fill], col[k], token);
        }
        token += kGroup;
        --left;
        fill = fill + 1 == kGroups ? 0 : fill + 1;
    }
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (i < left)
#pragma unroll
                for (int k = 0; k < N; ++k) next[i][k].load(src[k] + i * stride[k]);
        left -= kGroup;
#pragma unroll
        for (int k = 0; k < N; ++k) src[k] += kGroup * stride[k];
    }
    __device__ __forceinline__ void arrived() {
        if constexpr (BULK) wait_copy(&full[stage], parity, status, left);
    }
    // After the last get of a group: its place takes another.
    __device__ __forceinline__ void reuse() {
        if constexpr (BULK) {
            __syncwarp();
            issue();
            if (++stage == kGroups) stage = 0, parity ^= 1;
        }
    }
    // After the last group, before the block ends or its ring is used for something else.
    __device__ __forceinline__ void drain() const {
        if constexpr (BULK)
            if (threadIdx.x == 0) drain_ring(full, kGroups, stage, parity, left);
    }
    __device__ __forceinline__ void get(int i, int k, typename Lanes<VEC>::V* v) const {
        float f[VEC];
        if constexpr (BULK) {
            Pack<T, VEC> p;
            p.load(reinterpret_cast<const T*>(ring + (stage * N + k) * tile + i * line) +
                   threadIdx.x * VEC);
            p.get(f);
        } else {
            next[i][k].get(f);
        }
        to_lanes<VEC>(f, v);
    }
};

// The channels of a block: of one piece of the split only.
struct Channels {
    long long c0;   // first
    int n;          // how many
    int piece;
    int off;        // first channel within the piece
    long long c;    // this lane's first, or the block's where the lane has none
    bool on;        // this lane has channels
};
template <int VEC>
__device__ __forceinline__ Channels channels_of(const ConvArgs& a, int cb) {
    Channels r;
    r.piece = cb >= a.blk2 ? 2 : cb >= a.blk1 ? 1 : 0;
    const int first = r.piece == 2 ? a.blk2 : r.piece == 1 ? a.blk1 : 0;
    const int width = r.piece == 2 ? a.width[2] : r.piece == 1 ? a.width[1] : a.width[0];
    const int off = r.off = (cb - first) * (kLanes * VEC);
    r.c0 = (r.piece == 2 ? a.off2 : r.piece == 1 ? a.off1 : 0) + off;
    r.n = width - off < kLanes * VEC ? width - off : kLanes * VEC;
    r.on = (int)threadIdx.x * VEC < r.n;
    r.c = r.c0 + (r.on ? threadIdx.x * VEC : 0);
    return r;
}
// Token 0 of a piece's tensor at channel c of it.
template <typename T>
__device__ __forceinline__ T* piece_at(const ConvArgs& a, const Channels& ch, long long c, int* stride) {
    const int k = ch.piece;
    *stride = k == 2 ? a.width[2] : k == 1 ? a.width[1] : a.width[0];
    return static_cast<T*>(k == 2 ? a.out[2] : k == 1 ? a.out[1] : a.out[0]) +
           (c - (k == 2 ? a.off2 : k == 1 ? a.off1 : 0));
}

template <typename T, int VEC, int K>
__device__ __forceinline__ void token_lanes(const ConvArgs& a, const Seq& q, long long i, long long c,
                                            typename Lanes<VEC>::V* v) {
    float f[VEC];
    token<T, VEC, K>(a, q, i, c, f);
    to_lanes<VEC>(f, v);
}

// ------------------------------------------------------------------ forward
template <typename T, int VEC, int K, bool SILU>
__global__ void __launch_bounds__(kLanes* kRuns, 2) conv_fwd_kernel(const ConvArgs a, const __grid_constant__ ConvMaps maps) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    using In = Run<T, VEC, 1>;
    constexpr int kGroup = In::kGroup;
    __shared__ __align__(16) float ws[K + 1][kLanes * VEC];
    __shared__ RunBars bars;
    extern __shared__ __align__(128) char ring[];
    const int cb = blockIdx.x % a.nchblk, rb = blockIdx.x / a.nchblk;
    const Channels ch = channels_of<VEC>(a, cb);
    const long long c = ch.c;

    if (rb >= a.nrunblk) {  // the states: one (sequence, row) per thread row
        const long long item = (long long)(rb - a.nrunblk) * kRuns + threadIdx.y;
        if (!ch.on || item >= (long long)a.nseq * K) return;
        const Seq q = seq_at(a, (int)(item / K));
        const int r = (int)(item % K);
        const long long p0 = a.pos ? a.pos[q.s] : 0;
        const long long last = p0 + (q.end - q.start) - 1;
        const long long i = last - state_row<K>(last - r) - p0;  // token on row r: last such position
        float f[VEC];
        token<T, VEC, K>(a, q, i, c, f);
        store_vec<VEC>(static_cast<T*>(a.final_state) + item * a.C + c, f);
        return;
    }

    const long long t0 = ((long long)rb * kRuns + threadIdx.y) * a.run;
    const long long t1 = t0 + a.run < a.T ? t0 + a.run : a.T;
    In in;
    in.begin(t0, t0 < t1 ? (int)(t1 - t0) : 0, ring, &bars, a.status);
    if (t0 < t1 && (In::BULK || ch.on)) {  // on their way before the weights are looked at
        in.template tensor<0>(&maps.u, (int)ch.c0, static_cast<const T*>(a.u) + t0 * a.us + ch.c0, a.us);
        in.start();
    }
    stage_weights<VEC, K>(a, ch.c0, ch.n, ws);
    if (t0 >= t1 || (!In::BULK && !ch.on)) return;
    V w[K][N], b[N];
    to_lanes<VEC>(&ws[K][threadIdx.x * VEC], b);
#pragma unroll
    for (int k = 0; k < K; ++k) to_lanes<VEC>(&ws[k][threadIdx.x * VEC], w[k]);
    int ostride;
    T* out = piece_at<T>(a, ch, c, &ostride) + t0 * a.width[ch.piece];

    Seq q = seq_of(a, t0);
    V win[K - 1][N];  // win[j]: token t - 1 - j
#pragma unroll
    for (int j = 0; j < K - 1; ++j) token_lanes<T, VEC, K>(a, q, t0 - q.start - 1 - j, c, win[j]);

    const int total = (int)(t1 - t0);
    int end = near(q.end - t0);  // the sequence's end, from t0
    for (int n = 0; n < total; n += kGroup, out += kGroup * ostride) {
        in.arrived();
        V cur[kGroup][N];
        auto work = [&](int i, bool live) {
            V o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                V v = fma_(w[K - 1][e], cur[i][e], b[e]);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) v = fma_(w[K - 2 - j][e], win[j][e], v);
                o[e] = SILU ? mul_(v, sigmoid_lanes<T>(v)) : v;
#pragma unroll
                for (int j = K - 2; j > 0; --j) win[j][e] = win[j - 1][e];
                win[0][e] = cur[i][e];
            }
            float f[VEC];
            from_lanes<VEC>(o, f);
            if (!live)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = 0.f;
            if (ch.on) store_vec<VEC>(out + i * ostride, f);
        };
        const bool whole = n + kGroup <= total && n + kGroup <= end && q.live;  // the same for the warp
        if constexpr (!In::BULK) {  // the registers are read: the next group takes them
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                if (whole || n + i < total) in.get(i, 0, cur[i]);
            in.fetch();
        }
        if (whole) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                if constexpr (In::BULK) in.get(i, 0, cur[i]);
                work(i, true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                if (n + i >= total) break;
                if (n + i == end) {
                    q = seq_of(a, t0 + n + i);
                    end = near(q.end - t0);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) token_lanes<T, VEC, K>(a, q, -1 - j, c, win[j]);
                }
                if constexpr (In::BULK) in.get(i, 0, cur[i]);
                work(i, q.live);
            }
        }
        in.reuse();
    }
    in.drain();
}

// ------------------------------------------------------------------ backward
// g at one token: pre from the current token and its window.
template <typename T, int VEC, int K, bool SILU>
__device__ __forceinline__ void grad_pre(const typename Lanes<VEC>::V (*w)[Lanes<VEC>::N],
                                         const typename Lanes<VEC>::V* b,
                                         const typename Lanes<VEC>::V* cur,
                                         const typename Lanes<VEC>::V (*win)[Lanes<VEC>::N],
                                         const typename Lanes<VEC>::V* dy,
                                         typename Lanes<VEC>::V* g) {
    using V = typename Lanes<VEC>::V;
#pragma unroll
    for (int e = 0; e < Lanes<VEC>::N; ++e) {
        if constexpr (!SILU) {
            g[e] = dy[e];
            continue;
        }
        V v = fma_(w[K - 1][e], cur[e], b[e]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) v = fma_(w[K - 2 - j][e], win[j][e], v);
        const V s = sigmoid_lanes<T>(v);
        g[e] = mul_(dy[e], silu_slope(s, mul_(v, s)));
    }
}

// The carried state's gradient, row r of sequence q: from the first tokens that read the
// row's position p0 - m, and passed through where the row is still in the final state.
template <typename T, int VEC, int K, bool SILU>
__device__ __noinline__ void state_grad(const ConvArgs& a, const Seq& q, int r, long long c,
                                        const Channels& ch, const float (*ws)[kLanes * VEC]) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    V w[K][N], b[N];
    to_lanes<VEC>(&ws[K][threadIdx.x * VEC], b);
#pragma unroll
    for (int k = 0; k < K; ++k) to_lanes<VEC>(&ws[k][threadIdx.x * VEC], w[k]);
    const long long p0 = a.pos ? a.pos[q.s] : 0;
    const long long n = q.end - q.start;
    int m = state_row<K>(p0 - r);
    if (m == 0) m = K;
    const long long at = ((long long)q.s * K + r) * a.C + c;
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = 0.f;
    if (a.dfinal && m + n <= K) {
        Pack<T, VEC> v;
        v.load(static_cast<const T*>(a.dfinal) + at);
        v.get(f);
    }
    V d[N];
    to_lanes<VEC>(f, d);
    int dstride;
    const T* dout = piece_at<T>(a, ch, c, &dstride);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        if (i >= n || i + m >= K) break;
        V cur[N], win[K - 1][N], dy[N], g[N];
        token_lanes<T, VEC, K>(a, q, i, c, cur);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) token_lanes<T, VEC, K>(a, q, i - 1 - j, c, win[j]);
        Pack<T, VEC> v;
        v.load(dout + (q.start + i) * dstride);
        v.get(f);
        to_lanes<VEC>(f, dy);
        grad_pre<T, VEC, K, SILU>(w, b, cur, win, dy, g);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (k == K - 1 - (i + m))
#pragma unroll
                for (int e = 0; e < N; ++e) d[e] = fma_(w[k][e], g[e], d[e]);
    }
    from_lanes<VEC>(d, f);
    store_vec<VEC>(static_cast<T*>(a.dinit) + at, f);
}

template <typename T, int VEC, int K, bool SILU>
__global__ void __launch_bounds__(kLanes* kRuns, 2) conv_bwd_kernel(const ConvArgs a, const __grid_constant__ ConvMaps maps) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    using In = Run<T, VEC, 2>;
    constexpr int kGroup = In::kGroup;
    __shared__ __align__(16) float ws[K + 1][kLanes * VEC];
    __shared__ RunBars bars;
    extern __shared__ __align__(128) char ring[];
    const int cb = blockIdx.x % a.nchblk, rb = blockIdx.x / a.nchblk;
    const Channels ch = channels_of<VEC>(a, cb);
    const long long c = ch.c;

    if (rb >= a.nrunblk) {  // the carried states' gradients
        stage_weights<VEC, K>(a, ch.c0, ch.n, ws);
        const long long item = (long long)(rb - a.nrunblk) * kRuns + threadIdx.y;
        if (ch.on && item < (long long)a.nseq * K)
            state_grad<T, VEC, K, SILU>(a, seq_at(a, (int)(item / K)), (int)(item % K), c, ch, ws);
        return;
    }

    const long long t0 = ((long long)rb * kRuns + threadIdx.y) * a.run;
    const long long t1 = t0 + a.run < a.T ? t0 + a.run : a.T;
    // g of the K-1 tokens after the run reaches back into it
    const long long t2 = t1 + K - 1 < a.T ? t1 + K - 1 : a.T;
    const bool on = t0 < t1 && (In::BULK || ch.on);
    In in;
    in.begin(t0, t0 < t1 ? (int)(t2 - t0) : 0, ring, &bars, a.status);
    if (on) {
        int dstride;
        const T* dout = piece_at<T>(a, ch, ch.c0, &dstride);
        in.template tensor<0>(&maps.u, (int)ch.c0, static_cast<const T*>(a.u) + t0 * a.us + ch.c0, a.us);
        in.template tensor<1>(&maps.dout[ch.piece], ch.off, dout + t0 * dstride, dstride);
        in.start();
    }
    stage_weights<VEC, K>(a, ch.c0, ch.n, ws);
    V dw[K + 1][N];
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[k][e] = both<V>(0.f);

    if (on) {
        V w[K][N], b[N];
        to_lanes<VEC>(&ws[K][threadIdx.x * VEC], b);
#pragma unroll
        for (int k = 0; k < K; ++k) to_lanes<VEC>(&ws[k][threadIdx.x * VEC], w[k]);
        T* du = static_cast<T*>(a.du) + t0 * a.dus + c;  // token t of the loop below
        const long long dus = a.dus;
        Seq q = seq_of(a, t0);
        V win[K - 1][N];  // win[j]: token t - 1 - j
        V acc[K][N];      // acc[j]: du of token t - j so far
#pragma unroll
        for (int j = 0; j < K - 1; ++j) token_lanes<T, VEC, K>(a, q, t0 - q.start - 1 - j, c, win[j]);
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) acc[j][e] = both<V>(0.f);

        const int mine = (int)(t1 - t0), total = (int)(t2 - t0);
        int begin = near(q.start - t0), end = near(q.end - t0);  // the sequence, from t0
        for (int n = 0; n < total; n += kGroup, du += kGroup * dus) {
            in.arrived();
            V cur[kGroup][N], dy[kGroup][N], g[N];
            auto sums = [&](int i) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dw[K][e] = add_(dw[K][e], g[e]);
                    dw[K - 1][e] = fma_(g[e], cur[i][e], dw[K - 1][e]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j)
                        dw[K - 2 - j][e] = fma_(g[e], win[j][e], dw[K - 2 - j][e]);
                }
            };
            auto shift = [&](int i) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
#pragma unroll
                    for (int j = K - 2; j > 0; --j) win[j][e] = win[j - 1][e];
                    win[0][e] = cur[i][e];
                }
            };
            auto emit = [&](int i, const V* v) {  // token t0 + n + i
                float f[VEC];
                from_lanes<VEC>(v, f);
                if (ch.on) store_vec<VEC>(du + i * dus, f);
            };
            // a whole group inside the run, and no end or beginning of a sequence in reach; the
            // same for the warp
            const bool whole = n + kGroup <= mine && n + kGroup + K <= end && n >= begin + K - 1 && q.live;
            auto read = [&](int i) {
                in.get(i, 0, cur[i]);
                in.get(i, 1, dy[i]);
            };
            if constexpr (!In::BULK) {  // the registers are read: the next group takes them
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
                    if (whole || n + i < total) read(i);
                in.fetch();
            }
            if (whole) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    if constexpr (In::BULK) read(i);
                    grad_pre<T, VEC, K, SILU>(w, b, cur[i], win, dy[i], g);
                    sums(i);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
#pragma unroll
                        for (int j = K - 1; j > 0; --j)
                            acc[j][e] = fma_(w[K - 1 - j][e], g[e], acc[j - 1][e]);
                        acc[0][e] = mul_(w[K - 1][e], g[e]);
                    }
                    if (i >= K - 1 || n > 0) emit(i - (K - 1), acc[K - 1]);
                    shift(i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const int at = n + i;
                    if (at >= total) break;
                    if (at == end) {
                        q = seq_of(a, t0 + at);
                        begin = near(q.start - t0), end = near(q.end - t0);
#pragma unroll
                        for (int j = 0; j < K - 1; ++j)
                            token_lanes<T, VEC, K>(a, q, -1 - j, c, win[j]);
                    }
                    if constexpr (In::BULK) read(i);
                    grad_pre<T, VEC, K, SILU>(w, b, cur[i], win, dy[i], g);
                    if (!q.live)
#pragma unroll
                        for (int e = 0; e < N; ++e) g[e] = both<V>(0.f);
                    if (at < mine && q.live) sums(i);
                    // acc[j] becomes token at - j; token at starts from the final state's
                    // gradient where it is still in the window there
                    float f[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] = 0.f;
                    if (a.dfinal && q.live && end - at <= K) {
                        const long long p = (a.pos ? a.pos[q.s] : 0) + (t0 + at - q.start);
                        Pack<T, VEC> v;
                        v.load(static_cast<const T*>(a.dfinal) +
                               ((long long)q.s * K + state_row<K>(p)) * a.C + c);
                        v.get(f);
                    }
#pragma unroll
                    for (int j = K - 1; j > 0; --j)
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[j][e] = acc[j - 1][e];
                    to_lanes<VEC>(f, acc[0]);
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (at - j >= begin)  // a token of an earlier sequence gets nothing
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                acc[j][e] = fma_(w[K - 1 - j][e], g[e], acc[j][e]);
                    if (at >= K - 1) emit(i - (K - 1), acc[K - 1]);
                    shift(i);
                }
            }
            in.reuse();
        }
        // the last tokens of the run that nothing later reads
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const long long tok = t2 - 1 - j;
            if (ch.on && tok >= t0 && tok < t1) {
                float f[VEC];
                from_lanes<VEC>(acc[j], f);
                store_vec<VEC>(static_cast<T*>(a.du) + tok * dus + c, f);
            }
        }
    }

    // one partial per block, weight and channel: the runs are added in order, in the ring's place
    in.drain();
    float* red = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float f[VEC];
        from_lanes<VEC>(dw[k], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            red[((threadIdx.y * (K + 1) + k) * VEC + e) * kLanes + threadIdx.x] = f[e];
    }
    __syncthreads();
    for (int i = threadIdx.y * kLanes + threadIdx.x; i < (K + 1) * kLanes * VEC; i += kLanes * kRuns) {
        const int k = i / (kLanes * VEC), x = i - k * kLanes * VEC;
        if (x >= ch.n) continue;
        const int at = (k * VEC + x % VEC) * kLanes + x / VEC;
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < kRuns; ++y) s += red[y * (K + 1) * VEC * kLanes + at];
        a.partial[((long long)rb * (K + 1) + k) * a.C + ch.c0 + x] = s;
    }
}

// ------------------------------------------------------------------ host
struct Conv {
    long long T, C;
    int nseq;
    size_t e;
};

ssd_status_t check_conv(const ssd_conv_t* p, Conv* c) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->seqlen < 0 || p->nseq < 0) return SSD_ERR_INVALID_ARG;
    if (p->nseq > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
    if (!dtype_ok(p->dtype) || !dtype_ok(p->wdtype)) return SSD_ERR_INVALID_ARG;
    if (p->activation != 0 && p->activation != 1) return SSD_ERR_INVALID_ARG;
    long long C = 0;
    for (int i = 0; i < 3; ++i) {
        if (p->split[i] < 0 || (i > 0 && p->split[i] > 0 && p->split[i - 1] == 0))
            return SSD_ERR_INVALID_ARG;
        C += p->split[i];
    }
    if (C < 1) return SSD_ERR_INVALID_ARG;
    if (p->u_stride < C || (p->du_stride != 0 && p->du_stride < C)) return SSD_ERR_INVALID_ARG;
    if (p->width < 1) return SSD_ERR_INVALID_ARG;
    if (p->width < 2 || p->width > 4 || C > (1 << 24)) return SSD_ERR_UNSUPPORTED;
    if (p->seqlen > INT_MAX || p->batch > INT_MAX) return SSD_ERR_UNSUPPORTED;
    c->T = p->batch * p->seqlen;
    if (c->T > INT_MAX) return SSD_ERR_UNSUPPORTED;
    c->C = C;
    c->nseq = p->nseq > 0 ? p->nseq : (int)p->batch;
    c->e = dtype_size(p->dtype);
    return SSD_OK;
}

// Piece i of the outputs or of their gradients.
Span piece_span(const ssd_conv_t* p, const Conv& c, int i, const void* t) {
    return Span(t, c.T, p->split[i], p->split[i], c.e);
}

// Channels of a vector: `most` where every row of every tensor and every piece starts on 16
// bytes (and tokens move in bulk copies), else two or one.
int conv_vec(const ssd_conv_t* p, const Conv& c, int most, const void* const* ptrs, int np) {
    const long long strides[5] = {p->split[0], p->split[1], p->split[2], p->u_stride, p->du_stride};
    const int n = (int)(16 / c.e);
    bool wide = true, pairs = true;
    for (long long s : strides) wide = wide && s % n == 0, pairs = pairs && s % 2 == 0;
    for (int i = 0; i < np; ++i)
        wide = wide && aligned_to(ptrs[i], 16), pairs = pairs && aligned_to(ptrs[i], 2 * c.e);
    return wide ? most : pairs ? 2 : 1;
}
int most_fwd(const Conv& c) { return c.e == 2 ? 8 : 4; }
constexpr int kMostBwd = 4;  // 8 bytes of bf16: the sums take the registers of a wider vector

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Blocks of channels: none straddles two pieces.
int channel_blocks(const ssd_conv_t* p, int vec) {
    const int wide = kLanes * vec;
    return ceil_div(p->split[0], wide) + ceil_div(p->split[1], wide) + ceil_div(p->split[2], wide);
}

// Tokens a warp walks: the run with the shortest estimated time, which is the rounds of blocks
// (two an SM; three in short vectors) times a run and `over` tokens' worth of starting and
// ending it.  Few tokens get short runs, many the length that fills the last round: 65536
// tokens of 1792 channels took 90 us in runs of 64 (3.4 rounds).  Whole groups of eight tokens
// but for the shortest; `most` blocks along the tokens.
int choose_run(long long T, int nch, int vec, int over, long long most) {
    const long long at_once = (long long)sm_count() * (vec > 2 ? 2 : 3);
    long long best = -1;
    int pick = 1;
    for (long long run = 1; run <= (1 << 28); run = run < 8 ? run * 2 : run < 128 ? run + 8 : run * 2) {
        const long long nb = (T + run * kRuns - 1) / (run * kRuns);
        if (nb > most) continue;
        const long long cost = (nb * nch + at_once - 1) / at_once * (run + over);
        if (best >= 0 && cost >= best) {
            if (run >= 128) break;
            continue;
        }
        best = cost;
        pick = (int)run;
    }
    return pick;
}
int fwd_run(const ssd_conv_t* p, long long T, int vec) {
    return choose_run(T, channel_blocks(p, vec), vec, 8, 1LL << 40);
}
// Blocks along the tokens of the backward: the partial sums' count, and with it the workspace,
// follows it.
int bwd_run(const ssd_conv_t* p, long long T, int vec) {
    return choose_run(T, channel_blocks(p, vec), vec, 13, 1024);
}

void fill_args(const ssd_conv_t* p, const Conv& c, int vec, ConvArgs* a) {
    a->T = c.T;
    a->L = p->seqlen;
    a->C = c.C;
    a->us = p->u_stride;
    a->dus = p->du_stride;
    a->off1 = p->split[0];
    a->off2 = p->split[0] + p->split[1];
    for (int i = 0; i < 3; ++i) a->width[i] = p->split[i];
    const int wide = kLanes * vec;
    a->blk1 = ceil_div(p->split[0], wide);
    a->blk2 = a->blk1 + ceil_div(p->split[1], wide);
    a->nchblk = channel_blocks(p, vec);
    a->nseq = c.nseq;
    a->wbf16 = p->wdtype == SSD_DTYPE_BF16;
}

// Shared memory of a block: the ring, or in the backward the runs' sums at the end.
template <typename T, int VEC, int K>
constexpr size_t conv_smem(bool bwd) {
    const size_t n = bwd ? 2 : 1;
    const size_t ring = VEC >= 4 ? kRuns * n * kLanes * VEC * sizeof(T) * group_of(VEC, sizeof(T), n) *
                                       groups_of(VEC, sizeof(T), n)
                                 : 0;
    const size_t sums = bwd ? sizeof(float) * kRuns * (K + 1) * VEC * kLanes : 0;
    return ring > sums ? ring : sums;
}
// Map over a [rows][cols] tensor with rows `stride` elements apart: tiles of a group of
// rows and the columns of a block.
template <typename T, int VEC, int N>
bool make_tile_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long stride) {
    tcc::EncodeTiledFn enc = tcc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(stride * sizeof(T))};
    const cuuint32_t box[2] = {kLanes * VEC, (cuuint32_t)group_of(VEC, sizeof(T), N)};
    const cuuint32_t es[2] = {1, 1};
    return enc(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
               const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <bool BWD, typename T, int VEC, int K, bool SILU>
cudaError_t launch_k(unsigned grid, const ConvArgs& a, cudaStream_t s) {
    constexpr auto kernel = [] {
        if constexpr (BWD)
            return &conv_bwd_kernel<T, VEC, K, SILU>;
        else
            return &conv_fwd_kernel<T, VEC, K, SILU>;
    }();
    constexpr size_t smem = conv_smem<T, VEC, K>(BWD);
    ConvMaps maps;
    if (VEC >= 4 && a.T > 0) {
        if (!make_tile_map<T, VEC, BWD ? 2 : 1>(&maps.u, a.u, a.T, a.C, a.us)) return cudaErrorUnknown;
        for (int i = 0; BWD && i < 3; ++i)
            if (a.width[i] && !make_tile_map<T, VEC, BWD ? 2 : 1>(&maps.dout[i], a.out[i], a.T, a.width[i], a.width[i]))
                return cudaErrorUnknown;
    }
    const cudaError_t e = allow_smem<kernel>(smem);
    if (e == cudaSuccess) kernel<<<grid, dim3(kLanes, kRuns), smem, s>>>(a, maps);
    return e;
}
template <bool BWD, typename T, int VEC, bool SILU>
cudaError_t launch_vec(int K, unsigned grid, const ConvArgs& a, cudaStream_t s) {
    if (K == 2) return launch_k<BWD, T, VEC, 2, SILU>(grid, a, s);
    if (K == 3) return launch_k<BWD, T, VEC, 3, SILU>(grid, a, s);
    return launch_k<BWD, T, VEC, 4, SILU>(grid, a, s);
}
template <bool BWD, typename T, bool SILU>
cudaError_t launch_type(int vec, int K, unsigned grid, const ConvArgs& a, cudaStream_t s) {
    constexpr int wide = sizeof(T) == 2 && !BWD ? 8 : 4;
    if (vec == wide) return launch_vec<BWD, T, wide, SILU>(K, grid, a, s);
    if (vec == 2) return launch_vec<BWD, T, 2, SILU>(K, grid, a, s);
    return launch_vec<BWD, T, 1, SILU>(K, grid, a, s);
}
template <bool BWD, bool SILU>
cudaError_t launch_silu(const ssd_conv_t* p, int vec, unsigned grid, const ConvArgs& a, cudaStream_t s) {
    return p->dtype == SSD_DTYPE_BF16
               ? launch_type<BWD, __nv_bfloat16, SILU>(vec, p->width, grid, a, s)
               : launch_type<BWD, float, SILU>(vec, p->width, grid, a, s);
}
template <bool BWD>
cudaError_t launch_conv(const ssd_conv_t* p, int vec, unsigned grid, const ConvArgs& a, cudaStream_t s) {
    return p->activation == 1 ? launch_silu<BWD, true>(p, vec, grid, a, s)
                              : launch_silu<BWD, false>(p, vec, grid, a, s);
}

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" {

ssd_status_t ssd_conv_forward(const ssd_conv_t* conv, const void* u, const void* weight,
                              const void* bias, const int32_t* cu_seqlens,
                              const int32_t* positions, const void* initial_state, void* out0,
                              void* out1, void* out2, void* final_state, void* stream) {
    set_last_launches(0);
    Conv c;
    ssd_status_t st = check_conv(conv, &c);
    if (st != SSD_OK) return st;
    if ((conv->nseq > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    void* outs[3] = {out0, out1, out2};
    if (!weight) return SSD_ERR_INVALID_ARG;
    if (c.T > 0) {
        if (!u) return SSD_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            if (conv->split[i] && !outs[i]) return SSD_ERR_INVALID_ARG;
    }
    const void* ptrs[6] = {u, out0, out1, out2, initial_state, final_state};
    for (const void* p : ptrs)
        if (!aligned_to(p, c.e)) return SSD_ERR_ALIGNMENT;
    if (!aligned_to(weight, dtype_size(conv->wdtype)) ||
        !aligned_to(bias, dtype_size(conv->wdtype)) || !aligned_to(cu_seqlens, 4) ||
        !aligned_to(positions, 4))
        return SSD_ERR_ALIGNMENT;
    // a run reads tokens and states that other blocks may already have written over
    const long long srows = (long long)c.nseq * conv->width;
    if (clash({piece_span(conv, c, 0, out0), piece_span(conv, c, 1, out1), piece_span(conv, c, 2, out2),
               Span(final_state, srows * c.C, c.e)},
              {Span(u, c.T, conv->u_stride, c.C, c.e), Span(initial_state, srows * c.C, c.e),
               Span(weight, c.C * conv->width, dtype_size(conv->wdtype)),
               Span(bias, c.C, dtype_size(conv->wdtype)), Span(cu_seqlens, c.nseq + 1LL, 4),
               Span(positions, c.nseq, 4)}))
        return SSD_ERR_INVALID_ARG;
    if (c.T == 0 && !final_state) return SSD_OK;

    const int vec = conv_vec(conv, c, most_fwd(c), ptrs, 6);
    ConvArgs a = {};
    fill_args(conv, c, vec, &a);
    if (!(a.status = status_word())) return SSD_ERR_CUDA;
    a.u = u, a.w = weight, a.b = bias, a.cu = cu_seqlens, a.pos = positions;
    a.init = initial_state, a.final_state = final_state;
    for (int i = 0; i < 3; ++i) a.out[i] = outs[i];
    a.run = fwd_run(conv, c.T, vec);
    a.nrunblk = ceil_div(c.T, (long long)a.run * kRuns);
    const int nstate = final_state ? ceil_div(srows, kRuns) : 0;
    const long long grid = (long long)a.nchblk * (a.nrunblk + nstate);
    if (grid > INT_MAX) return SSD_ERR_UNSUPPORTED;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("conv_fwd");
    cudaError_t e = launch_conv<false>(conv, vec, (unsigned)grid, a, L.stream);
    const cudaError_t last = L.end();
    if (e == cudaSuccess) e = last;
    set_last_launches(L.count);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_conv_workspace_size(const ssd_conv_t* conv, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    Conv c;
    ssd_status_t st = check_conv(conv, &c);
    if (st != SSD_OK) return st;
    size_t most = 0;
    for (int vec = kMostBwd; vec >= 1; vec = vec > 2 ? 2 : vec - 1) {  // any may run, by the pointers' alignment
        const int nb = ceil_div(c.T, (long long)bwd_run(conv, c.T, vec) * kRuns);
        const size_t n = sizeof(float) * (size_t)nb * (conv->width + 1) * c.C;
        if (n > most) most = n;
    }
    *bytes = most > 256 ? (most + 255) / 256 * 256 : 256;
    return SSD_OK;
}

ssd_status_t ssd_conv_backward(const ssd_conv_t* conv, const void* u, const void* weight,
                               const void* bias, const int32_t* cu_seqlens,
                               const int32_t* positions, const void* initial_state,
                               const void* dout0, const void* dout1, const void* dout2,
                               const void* d_final_state, void* du, void* d_weight, void* d_bias,
                               void* d_initial_state, void* workspace, size_t workspace_bytes,
                               void* stream) {
    set_last_launches(0);
    Conv c;
    ssd_status_t st = check_conv(conv, &c);
    if (st != SSD_OK) return st;
    if ((conv->nseq > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const void* douts[3] = {dout0, dout1, dout2};
    if (!weight || !d_weight || (d_bias && !bias)) return SSD_ERR_INVALID_ARG;
    if (conv->du_stride == 0) return SSD_ERR_INVALID_ARG;
    if (c.T > 0) {
        if (!u || !du) return SSD_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            if (conv->split[i] && !douts[i]) return SSD_ERR_INVALID_ARG;
    }
    const void* ptrs[8] = {u, dout0, dout1, dout2, initial_state, d_final_state, du, d_initial_state};
    for (const void* p : ptrs)
        if (!aligned_to(p, c.e)) return SSD_ERR_ALIGNMENT;
    const size_t we = dtype_size(conv->wdtype);
    if (!aligned_to(weight, we) || !aligned_to(bias, we) || !aligned_to(d_weight, we) ||
        !aligned_to(d_bias, we) || !aligned_to(cu_seqlens, 4) || !aligned_to(positions, 4))
        return SSD_ERR_ALIGNMENT;
    const long long srows = (long long)c.nseq * conv->width;
    size_t need = 0;
    st = ssd_conv_workspace_size(conv, &need);
    if (st != SSD_OK) return st;
    if (clash({Span(du, c.T, conv->du_stride, c.C, c.e), Span(d_weight, c.C * conv->width, we),
               Span(d_bias, c.C, we), Span(d_initial_state, srows * c.C, c.e), Span(workspace, need, 1)},
              {Span(u, c.T, conv->u_stride, c.C, c.e), piece_span(conv, c, 0, dout0),
               piece_span(conv, c, 1, dout1), piece_span(conv, c, 2, dout2),
               Span(initial_state, srows * c.C, c.e), Span(d_final_state, srows * c.C, c.e),
               Span(weight, c.C * conv->width, we), Span(bias, c.C, we),
               Span(cu_seqlens, c.nseq + 1LL, 4), Span(positions, c.nseq, 4)}))
        return SSD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;

    const int vec = conv_vec(conv, c, kMostBwd, ptrs, 8);
    ConvArgs a = {};
    fill_args(conv, c, vec, &a);
    if (!(a.status = status_word())) return SSD_ERR_CUDA;
    a.u = u, a.w = weight, a.b = bias, a.cu = cu_seqlens, a.pos = positions;
    a.init = initial_state, a.dfinal = d_final_state, a.du = du, a.dinit = d_initial_state;
    for (int i = 0; i < 3; ++i) a.out[i] = const_cast<void*>(douts[i]);
    a.partial = static_cast<float*>(workspace);
    a.run = bwd_run(conv, c.T, vec);
    a.nrunblk = ceil_div(c.T, (long long)a.run * kRuns);
    const int nstate = d_initial_state ? ceil_div(srows, kRuns) : 0;
    const long long grid = (long long)a.nchblk * (a.nrunblk + nstate);
    if (grid > INT_MAX) return SSD_ERR_UNSUPPORTED;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (grid > 0) {
        L.begin("conv_bwd");
        e = launch_conv<true>(conv, vec, (unsigned)grid, a, L.stream);
        const cudaError_t last = L.end();
        if (e == cudaSuccess) e = last;
    }
    if (e == cudaSuccess) {
        ReduceDst d = {};
        for (int k = 0; k < conv->width; ++k) {
            d.dst[k] = static_cast<char*>(d_weight) + k * we;
            d.step[k] = conv->width;
        }
        d.dst[conv->width] = d_bias;
        d.step[conv->width] = 1;
        e = launch_partial_sum(a.partial, a.nrunblk, conv->width + 1, c.C, d, conv->wdtype, L);
    }
    set_last_launches(L.count);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
