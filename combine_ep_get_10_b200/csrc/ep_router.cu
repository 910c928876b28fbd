// ep_router.cu -- the token router, its balance losses and their gradient.
//
// All kernels give a token's row of E <= 1024 logits to one warp and keep it in
// registers: lane L holds the NPL consecutive logits from e0(L) on, so that
// lane order is expert order (a tie is settled by the lowest lane) and, with
// groups, a group is a run of whole lanes.
#include <algorithm>
#include <cfloat>

#include "ep_device.cuh"
#include "ep_router_launch.h"

namespace ep {

namespace {

constexpr int kTopkWarps = 4;
constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------------ rows
// The lane's run of experts: [e0, e0 + n), n <= c <= NPL.  G (a power of two)
// groups take 32 / G lanes each; G = 1 spreads the row over all lanes.
struct LaneRun {
    int e0, n;
};

__host__ __device__ __forceinline__ int run_length(int E, int G)
{
    const int lanes = 32 / G;
    return (E / G + lanes - 1) / lanes;
}

__device__ __forceinline__ LaneRun lane_run(int E, int G, int lane)
{
    const int lanes = 32 / G, per = E / G, c = run_length(E, G);
    const int g = lane / lanes, q = lane - g * lanes;
    return {g * per + min(q * c, per), max(0, min(c, per - q * c))};
}

// A logit as the operators take it: NaN closes the expert like -inf, values
// above the largest finite one count as that one (so that l - max is never
// inf - inf).
__device__ __forceinline__ float clean_logit(float l)
{
    return l > kNegInf ? fminf(l, FLT_MAX) : kNegInf;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i)
{
    if (BF16)
        return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(logits) + i)) << 16);
    return __ldg(static_cast<const float*>(logits) + i);
}

// The lane's logits, closed ones and the places past its run as -inf.  vec:
// every lane has NPL of them and the rows are aligned for vector loads.
template <int NPL, bool BF16>
__device__ __forceinline__ void load_row(float (&v)[NPL], const void* logits, int64_t row, int E, LaneRun r, bool vec)
{
    const int64_t at = row * E + r.e0;
    if (vec && !BF16 && NPL % 4 == 0) {
#pragma unroll
        for (int j = 0; j < NPL / 4; ++j) {
            const uint4 w = ld_nc_v4(static_cast<const float*>(logits) + at + 4 * j);
            v[4 * j + 0] = __uint_as_float(w.x);
            v[4 * j + 1] = __uint_as_float(w.y);
            v[4 * j + 2] = __uint_as_float(w.z);
            v[4 * j + 3] = __uint_as_float(w.w);
        }
    } else if (vec && BF16 && NPL % 8 == 0) {
#pragma unroll
        for (int j = 0; j < NPL / 8; ++j) {
            const uint4 w = ld_nc_v4(static_cast<const uint16_t*>(logits) + at + 8 * j);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[8 * j + 2 * i] = bf16_lo(u[i]);
                v[8 * j + 2 * i + 1] = bf16_hi(u[i]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            v[j] = j < r.n ? load_logit<BF16>(logits, at + j) : kNegInf;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        v[j] = clean_logit(v[j]);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kFullMask, v, d));
    return v;
}

__device__ __forceinline__ float warp_min(float v)
{
    return -warp_max(-v);
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v += __shfl_xor_sync(kFullMask, v, d);
    return v;
}

template <int NPL>
__device__ __forceinline__ float row_max(const float (&v)[NPL])
{
    float m = v[0];
#pragma unroll
    for (int j = 1; j < NPL; ++j)
        m = fmaxf(m, v[j]);
    return warp_max(m);
}

__device__ __forceinline__ float sigmoid(float l)
{
    return 1.0f / (1.0f + expf(-l));
}

// Below this, sigmoid(l) = exp(l) to fp32 precision, and ratios of sigmoids are
// taken as ratios of exponentials, which do not underflow.
constexpr float kSigmoidTail = -60.0f;

// -------------------------------------------------------------- selection
// Finite floats and +inf as unsigned integers of the same order; 0 is below
// every one of them and stands for "cannot be chosen".  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float c)
{
    const uint32_t b = __float_as_uint(c + 0.0f);
    return b ^ ((b >> 31) != 0u ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) != 0u ? 0x80000000u : 0xffffffffu));
}

// The choice of one row in fp64, for the rows whose fp32 values lie too close
// together to tell their order.  c (shared memory of this warp): E values.
// Lane k returns the k-th chosen id, or -1.
template <bool BF16>
__device__ __noinline__ int choose_wide(const RouterTopkLaunch& a, int64_t row, double* c, int lane)
{
    const int E = a.r.num_experts, K = a.r.num_topk, G = a.r.num_groups;
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const double none = -INFINITY;
    double m = none, z = 0.0;
    if (softmax) {
        for (int e = lane; e < E; e += 32)
            m = fmax(m, static_cast<double>(clean_logit(load_logit<BF16>(a.logits, row * E + e))));
        for (int d = 16; d >= 1; d >>= 1)
            m = fmax(m, __shfl_xor_sync(kFullMask, m, d));
        for (int e = lane; e < E; e += 32) {
            const double l = clean_logit(load_logit<BF16>(a.logits, row * E + e));
            if (l > none)
                z += exp(l - m);
        }
        for (int d = 16; d >= 1; d >>= 1)
            z += __shfl_xor_sync(kFullMask, z, d);
    }
    for (int e = lane; e < E; e += 32) {
        const double l = clean_logit(load_logit<BF16>(a.logits, row * E + e));
        double v = none;
        if (l > none) {
            v = softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l));
            v += a.bias != nullptr ? static_cast<double>(__ldg(a.bias + e)) : 0.0;
            if (!(v > none))
                v = none; // a bias of -inf or NaN
        }
        c[e] = v;
    }
    __syncwarp();
    if (G > 1) {
        const int per = E / G;
        double mine = none; // lane g: the value of group g
        for (int g = 0; g < G; ++g) {
            double t1 = none, t2 = none;
            for (int e = lane; e < per; e += 32) {
                const double v = c[g * per + e];
                t2 = fmax(t2, fmin(t1, v));
                t1 = fmax(t1, v);
            }
            for (int d = 16; d >= 1; d >>= 1) {
                const double o1 = __shfl_xor_sync(kFullMask, t1, d), o2 = __shfl_xor_sync(kFullMask, t2, d);
                t2 = fmax(fmin(t1, o1), fmax(t2, o2));
                t1 = fmax(t1, o1);
            }
            if (lane == g)
                mine = a.r.group_top == 2 && t2 > none ? t1 + t2 : t1;
        }
        int before = 0;
        for (int g = 0; g < G; ++g) {
            const double o = __shfl_sync(kFullMask, mine, g);
            before += (o > mine || (o == mine && g < lane)) ? 1 : 0;
        }
        const uint32_t kept = __ballot_sync(kFullMask, lane < G && before < a.r.topk_groups);
        for (int e = lane; e < E; e += 32)
            if (((kept >> (e / per)) & 1u) == 0u)
                c[e] = none;
        __syncwarp();
    }
    int chosen = -1;
    for (int k = 0; k < K; ++k) {
        double best = none;
        int at = E;
        for (int e = lane; e < E; e += 32) {
            const double v = c[e];
            if (v > best) {
                best = v;
                at = e;
            }
        }
        for (int d = 16; d >= 1; d >>= 1) {
            const double o = __shfl_xor_sync(kFullMask, best, d);
            const int oi = __shfl_xor_sync(kFullMask, at, d);
            if (o > best || (o == best && oi < at)) {
                best = o;
                at = oi;
            }
        }
        if (at >= E)
            break;
        if (lane == k)
            chosen = at;
        __syncwarp();
        if (lane == 0)
            c[at] = none;
        __syncwarp();
    }
    return chosen;
}

// One warp a token.  Without bias and groups the choice is by the logits
// themselves and exact.  Otherwise the fp32 values c carry an error of at most
// err(c): half an ulp of the sum with the bias, and that of s,
//   sigmoid: expf 2 ulp, the sum and the quotient half an ulp each, on s <= 1:
//            6 * 2^-24 < 5e-7;
//   softmax: l - max half an ulp of it (times p <= exp(l - max) / Z: at most
//            0.37 / Z), expf 2 ulp, the sum of E terms NPL + 5 roundings and the
//            same again inside, on p <= 1 / Z: less than 64 * 2^-24 / Z;
// a row whose order those errors could change (adjacent chosen values, the last
// chosen one and the next, the last group kept and the first one dropped) is
// chosen again in fp64.  Values that are equal because logit and bias are
// equal need no second look.
template <int NPL, bool BF16>
__global__ void __launch_bounds__(kTopkWarps * 32) router_topk_kernel(RouterTopkLaunch a, bool vec)
{
    extern __shared__ double s_wide[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp;
    if (t >= a.r.num_tokens)
        return;
    const int E = a.r.num_experts, K = a.r.num_topk, G = a.r.num_groups;
    int64_t* idx_out = a.topk_idx + t * K;
    float* w_out = a.topk_weights + t * K;
    if (a.token_mask != nullptr && __ldg(a.token_mask + t) == 0) {
        if (lane < K) {
            idx_out[lane] = -1;
            w_out[lane] = 0.0f;
        }
        return;
    }
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const bool by_logit = a.bias == nullptr && G == 1;
    const LaneRun r = lane_run(E, G, lane);
    float v[NPL];
    load_row<NPL, BF16>(v, a.logits, t, E, r, vec);

    float m = 0.0f, z = 1.0f;
    if (softmax && (!by_logit || a.r.normalize == 0)) {
        m = row_max(v);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            sum += v[j] > kNegInf ? expf(v[j] - m) : 0.0f;
        z = warp_sum(sum);
    }
    const float es = softmax ? 4e-6f / z : 5e-7f;
    const auto err = [es](float c) { return es + 1.3e-7f * fabsf(c); };
    bool sure = true;
    uint32_t key[NPL];
    if (by_logit) {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            key[j] = v[j] > kNegInf ? order_key(v[j]) : 0u;
    } else {
        float c[NPL];
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            float s = softmax ? expf(v[j] - m) / z : sigmoid(v[j]);
            if (a.bias != nullptr && j < r.n)
                s += __ldg(a.bias + r.e0 + j);
            c[j] = v[j] > kNegInf && s > kNegInf ? s : kNegInf;
        }
        bool stay = true;
        if (G > 1 && a.r.topk_groups < G) {
            const int lanes = 32 / G, mine = lane / lanes;
            float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                t2 = fmaxf(t2, fminf(t1, c[j]));
                t1 = fmaxf(t1, c[j]);
            }
            for (int d = lanes >> 1; d >= 1; d >>= 1) {
                const float o1 = __shfl_xor_sync(kFullMask, t1, d), o2 = __shfl_xor_sync(kFullMask, t2, d);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            const bool two = a.r.group_top == 2 && t2 > kNegInf;
            const float value = two ? t1 + t2 : t1;
            const float ge = err(t1) + (two ? err(t2) : 0.0f) + 1.3e-7f * fabsf(value);
            int before = 0;
            for (int g = 0; g < G; ++g) {
                const float o = __shfl_sync(kFullMask, value, g * lanes);
                before += (o > value || (o == value && g < mine)) ? 1 : 0;
            }
            stay = before < a.r.topk_groups;
            const float low = warp_min(stay ? value - ge : INFINITY);
            const float high = warp_max(stay || value == kNegInf ? kNegInf : value + ge);
            sure = high == kNegInf || low > high;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            key[j] = stay && c[j] > kNegInf ? order_key(c[j]) : 0u;
    }

    // the K largest, in order, one a step: lane k keeps the k-th; the check
    // needs the one after them too
    int my_idx = -1, next_idx = -1;
    uint32_t my_key = 0u, next_key = 0u;
    const int steps = by_logit ? K : K + 1;
    for (int k = 0; k < steps; ++k) {
        uint32_t best = 0u;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (key[j] > best) {
                best = key[j];
                bj = j;
            }
        const uint32_t top = __reduce_max_sync(kFullMask, best);
        if (top == 0u)
            break;
        const int from = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int e = __shfl_sync(kFullMask, r.e0 + bj, from);
        if (lane == from) {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j == bj)
                    key[j] = 0u;
        }
        if (lane == k) {
            my_idx = e;
            my_key = top;
        }
        if (k == K) {
            next_idx = e;
            next_key = top;
        }
    }
    if (!by_logit && sure) {
        const float l = my_idx >= 0 ? clean_logit(load_logit<BF16>(a.logits, t * E + my_idx)) : 0.0f;
        const float b = my_idx >= 0 && a.bias != nullptr ? __ldg(a.bias + my_idx) : 0.0f;
        uint32_t nk = __shfl_down_sync(kFullMask, my_key, 1);
        float nl = __shfl_down_sync(kFullMask, l, 1), nb = __shfl_down_sync(kFullMask, b, 1);
        if (lane == K - 1) {
            nk = next_key;
            if (next_idx >= 0) {
                nl = clean_logit(load_logit<BF16>(a.logits, t * E + next_idx));
                nb = a.bias != nullptr ? __ldg(a.bias + next_idx) : 0.0f;
            }
        }
        bool apart = true;
        if (lane < K && nk != 0u) {
            const float c = key_value(my_key), n = key_value(nk);
            apart = c - err(c) > n + err(n) || (l == nl && b == nb);
        }
        sure = __all_sync(kFullMask, apart);
    }
    if (!sure)
        my_idx = choose_wide<BF16>(a, t, s_wide + static_cast<size_t>(warp) * E, lane);
    else if (lane >= K)
        my_idx = -1;

    const bool got = my_idx >= 0;
    const float l = got ? clean_logit(load_logit<BF16>(a.logits, t * E + my_idx)) : kNegInf;
    float w = 0.0f;
    if (a.r.normalize != 0) {
        const float lm = warp_max(l);
        if (got)
            w = softmax || lm < kSigmoidTail ? expf(l - lm) : sigmoid(l);
        const float total = warp_sum(w);
        w = got ? w / total : 0.0f;
    } else if (got) {
        w = softmax ? expf(l - m) / z : sigmoid(l);
    }
    if (lane < K) {
        idx_out[lane] = my_idx;
        w_out[lane] = a.r.scale * w;
    }
}

// ------------------------------------------------------------ balance loss
// Tokens are dealt out in chunks of at most kChunk tokens of one sequence,
// sequence after sequence: a CTA sums one chunk into its own partial row, and
// a second kernel sums each sequence's partial rows in order (fixed order, no
// floating-point atomics).
constexpr int kChunk = 64;
constexpr int kBalanceWarps = 8;

__host__ __device__ __forceinline__ int64_t balance_items(int64_t T, int64_t S)
{
    return (T + kChunk - 1) / kChunk + S; // at most one part chunk a sequence
}

struct BalancePartials {
    float* q;     // [items, E]
    int32_t* cnt; // [items, E]
    float* z;     // [items]
    int32_t* n;   // [items]
};

__host__ __device__ __forceinline__ BalancePartials balance_partials(void* workspace, int64_t items, int64_t E)
{
    float* q = static_cast<float*>(workspace);
    int32_t* cnt = reinterpret_cast<int32_t*>(q + items * E);
    float* z = reinterpret_cast<float*>(cnt + items * E);
    return {q, cnt, z, reinterpret_cast<int32_t*>(z + items)};
}

struct TokenRange {
    int begin, end;
};

// Tokens of sequence s; offsets are clamped so that bad ones stay in bounds.
__device__ __forceinline__ TokenRange seq_range(const int32_t* offsets, int T, int s)
{
    if (offsets == nullptr)
        return {0, T};
    const int b = min(max(__ldg(offsets + s), 0), T);
    return {b, min(max(__ldg(offsets + s + 1), b), T)};
}

// Chunks of the sequences before s, for s = S all of them; one warp, lanes agree.
__device__ __forceinline__ int64_t chunks_before(const int32_t* offsets, int T, int s, int lane)
{
    int64_t total = 0;
    for (int base = 0; base < s; base += 32) {
        int n = 0;
        if (base + lane < s) {
            const TokenRange r = seq_range(offsets, T, base + lane);
            n = (r.end - r.begin + kChunk - 1) / kChunk;
        }
        total += __reduce_add_sync(kFullMask, n);
    }
    return total;
}

// The sequence and chunk of item i; false when there are fewer items.
__device__ __forceinline__ bool find_chunk(const int32_t* offsets, int T, int S, int64_t i, int lane, int& seq,
                                           TokenRange& tokens)
{
    int64_t before = 0;
    for (int base = 0; base < S; base += 32) {
        int n = 0;
        if (base + lane < S) {
            const TokenRange r = seq_range(offsets, T, base + lane);
            n = (r.end - r.begin + kChunk - 1) / kChunk;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kFullMask, inc, d);
            if (lane >= d)
                inc += o;
        }
        const uint32_t past = __ballot_sync(kFullMask, before + inc > i);
        if (past != 0u) {
            const int l = __ffs(past) - 1;
            const int64_t first = before + __shfl_sync(kFullMask, inc - n, l);
            seq = base + l;
            const TokenRange r = seq_range(offsets, T, seq);
            tokens.begin = r.begin + static_cast<int>(i - first) * kChunk;
            tokens.end = min(r.end, tokens.begin + kChunk);
            return true;
        }
        before += __shfl_sync(kFullMask, inc, 31);
    }
    return false;
}

template <int NPL, bool BF16>
__global__ void __launch_bounds__(kBalanceWarps * 32) balance_chunk_kernel(BalanceLaunch a, bool vec)
{
    extern __shared__ float s_q[]; // [kBalanceWarps, E] sums, then [E] counts
    __shared__ float s_z[kBalanceWarps];
    __shared__ int s_n[kBalanceWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.r.num_experts, K = a.r.num_topk, T = a.r.num_tokens;
    int32_t* s_cnt = reinterpret_cast<int32_t*>(s_q + kBalanceWarps * E);
    int seq;
    TokenRange tokens;
    if (!find_chunk(a.seq_offsets, T, a.num_seqs, blockIdx.x, lane, seq, tokens))
        return; // the whole CTA: every warp sees the same answer
    for (int e = tid; e < E; e += blockDim.x)
        s_cnt[e] = 0;
    __syncthreads();

    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const LaneRun r = lane_run(E, 1, lane);
    float acc[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        acc[j] = 0.0f;
    float zz = 0.0f;
    int live = 0;
    for (int t = tokens.begin + warp; t < tokens.end; t += kBalanceWarps) {
        if (a.token_mask != nullptr && __ldg(a.token_mask + t) == 0)
            continue;
        float v[NPL];
        load_row<NPL, BF16>(v, a.logits, t, E, r, vec);
        const float m = row_max(v);
        if (!(m > kNegInf))
            continue; // every expert closed
        if (lane < K) {
            const int64_t e = __ldg(a.topk_idx + static_cast<int64_t>(t) * K + lane);
            if (e >= 0 && e < E)
                atomicAdd(s_cnt + e, 1);
        }
        ++live;
        float sum = 0.0f;
        float p[NPL];
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            p[j] = v[j] > kNegInf ? expf(v[j] - m) : 0.0f;
            sum += p[j];
        }
        sum = warp_sum(sum);
        const float lse = m + logf(sum);
        zz += lse * lse;
        if (!softmax && m >= kSigmoidTail) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                p[j] = v[j] > kNegInf ? sigmoid(v[j]) : 0.0f;
                sum += p[j];
            }
            sum = warp_sum(sum);
        }
        const float inv = 1.0f / sum;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            acc[j] += p[j] * inv;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        if (j < r.n)
            s_q[warp * E + r.e0 + j] = acc[j];
    if (lane == 0) {
        s_z[warp] = zz;
        s_n[warp] = live;
    }
    __syncthreads();
    const BalancePartials part = balance_partials(a.workspace, balance_items(T, a.num_seqs), E);
    const int64_t item = blockIdx.x;
    for (int e = tid; e < E; e += blockDim.x) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalanceWarps; ++w)
            sum += s_q[w * E + e];
        part.q[item * E + e] = sum;
        part.cnt[item * E + e] = s_cnt[e];
    }
    if (tid == 0) {
        float z = 0.0f;
        int n = 0;
        for (int w = 0; w < kBalanceWarps; ++w) {
            z += s_z[w];
            n += s_n[w];
        }
        part.z[item] = z;
        part.n[item] = n;
    }
}

// One CTA a sequence: its chunks' partial rows summed, then the losses.  The
// CTA's threads are `slices` runs of E (rounded up to whole warps); each run
// sums every slices-th chunk, and the runs are added in order.
constexpr int kFinishThreads = 1024;

__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(BalanceLaunch a)
{
    __shared__ float s_sum[kFinishThreads];
    __shared__ int s_cnt[kFinishThreads];
    __shared__ float s_red[kFinishThreads / 32];
    __shared__ int s_tokens;
    __shared__ float s_zsum;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.r.num_experts, T = a.r.num_tokens, s = blockIdx.x;
    const int64_t items = balance_items(T, a.num_seqs);
    const BalancePartials part = balance_partials(a.workspace, items, E);
    const int64_t i0 = min(items, chunks_before(a.seq_offsets, T, s, lane));
    const TokenRange tokens = seq_range(a.seq_offsets, T, s);
    const int64_t i1 = min(items, i0 + (tokens.end - tokens.begin + kChunk - 1) / kChunk);
    if (warp == 0) {
        int n = 0;
        float z = 0.0f;
        for (int64_t i = i0 + lane; i < i1; i += 32) {
            n += part.n[i];
            z += part.z[i];
        }
        n = __reduce_add_sync(kFullMask, n);
        z = warp_sum(z);
        if (lane == 0) {
            s_tokens = n;
            s_zsum = z;
        }
    }
    const int width = (E + 31) / 32 * 32;
    const int slices = kFinishThreads / width;
    const int e = tid % width, slice = tid / width;
    float q = 0.0f;
    int cnt = 0;
    if (e < E && slice < slices) {
#pragma unroll 8
        for (int64_t i = i0 + slice; i < i1; i += slices) {
            q += part.q[i * E + e];
            cnt += part.cnt[i * E + e];
        }
    }
    s_sum[tid] = q;
    s_cnt[tid] = cnt;
    __syncthreads();
    const int n = s_tokens;
    float fp = 0.0f;
    if (tid < E) {
        for (int i = 1; i < slices; ++i) {
            q += s_sum[i * width + tid];
            cnt += s_cnt[i * width + tid];
        }
        const float mean = n > 0 ? q / static_cast<float>(n) : 0.0f;
        a.counts[static_cast<int64_t>(s) * E + tid] = cnt;
        if (a.mean_scores != nullptr)
            a.mean_scores[static_cast<int64_t>(s) * E + tid] = mean;
        fp = static_cast<float>(cnt) * mean;
    }
    fp = warp_sum(fp);
    if (lane == 0)
        s_red[warp] = fp;
    __syncthreads();
    if (warp == 0) {
        fp = warp_sum(s_red[lane]);
        if (lane == 0) {
            const float nf = static_cast<float>(n);
            a.losses[2 * s] = n > 0 ? fp * (static_cast<float>(E) / (static_cast<float>(a.r.num_topk) * nf)) : 0.0f;
            a.losses[2 * s + 1] = n > 0 ? s_zsum / nf : 0.0f;
            a.seq_tokens[s] = n;
        }
    }
}

// ---------------------------------------------------------------- backward
constexpr int kBackwardWarps = 4;

// The sequence of token t (the last one that begins at or before it), -1 when
// it is in none: each step reads 32 offsets spread over what is left.
__device__ __forceinline__ int find_seq(const int32_t* offsets, int S, int t, int lane)
{
    if (offsets == nullptr)
        return 0;
    int lo = 0, len = S + 1; // how many of the S + 1 offsets are <= t: lo of them so far
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int at = lo + (lane + 1) * step - 1; // the last one of the lane's run
        const bool le = at < lo + len && __ldg(offsets + at) <= t;
        const int runs = __popc(__ballot_sync(kFullMask, le));
        lo += runs * step;
        if (step == 1)
            break;
        len = min(step - 1, S + 1 - lo);
    }
    const int s = lo - 1;
    return s < S ? s : -1;
}

template <int NPL, bool BF16>
__global__ void __launch_bounds__(kBackwardWarps * 32) router_backward_kernel(RouterBackwardLaunch a, bool vec)
{
    extern __shared__ float s_add[]; // [kBackwardWarps, E]: the chosen experts' part
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kBackwardWarps + warp;
    if (t >= a.r.num_tokens)
        return;
    const int E = a.r.num_experts, K = a.r.num_topk;
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const LaneRun r = lane_run(E, 1, lane);
    float* add = s_add + static_cast<size_t>(warp) * E;

    float d[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        d[j] = 0.0f;
    const bool on = a.token_mask == nullptr || __ldg(a.token_mask + t) != 0;
    float v[NPL];
    float m = kNegInf;
    if (on) {
        load_row<NPL, BF16>(v, a.logits, t, E, r, vec);
        m = row_max(v);
    }
    if (m > kNegInf) {
        // softmax of the row
        float p[NPL];
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            p[j] = v[j] > kNegInf ? expf(v[j] - m) : 0.0f;
            z += p[j];
        }
        z = warp_sum(z);
        const float inv_z = 1.0f / z;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            p[j] *= inv_z;

        if (a.d_topk_weights != nullptr) {
            // lane k: slot k's expert, logit and gradient
            int64_t e = -1;
            float l = kNegInf, g = 0.0f;
            if (lane < K) {
                e = __ldg(a.topk_idx + t * K + lane);
                if (e >= 0 && e < E)
                    l = clean_logit(load_logit<BF16>(a.logits, t * E + e));
            }
            const bool got = l > kNegInf;
            if (got)
                g = a.r.scale * __ldg(a.d_topk_weights + t * K + lane);
            float part = 0.0f; // what slot k adds at its expert
            float through = 0.0f; // softmax without normalize: sum of g p, for the whole row
            if (a.r.normalize != 0) {
                const float lm = warp_max(l);
                const bool tail = lm < kSigmoidTail;
                float w = got ? (softmax || tail ? expf(l - lm) : sigmoid(l)) : 0.0f;
                const float total = warp_sum(w);
                w = got ? w / total : 0.0f;
                const float mean = warp_sum(g * w);
                part = w * (g - mean);
                if (!softmax && got)
                    part *= 1.0f / (1.0f + expf(l)); // 1 - s
            } else if (softmax) {
                part = got ? g * (expf(l - m) * inv_z) : 0.0f;
                through = warp_sum(part);
            } else if (got) {
                part = g * sigmoid(l) * (1.0f / (1.0f + expf(l)));
            }
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j < r.n)
                    add[r.e0 + j] = 0.0f;
            __syncwarp();
            // slots of one expert (a caller's own ids) are added in slot order
            const uint32_t same = __match_any_sync(kFullMask, got ? static_cast<int>(e) : -1 - lane);
            if (__all_sync(kFullMask, __popc(same) == 1)) {
                if (got)
                    add[e] = part;
            } else {
                for (int k = 0; k < K; ++k) {
                    if (lane == k && got)
                        add[e] += part;
                    __syncwarp();
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j < r.n)
                    d[j] = add[r.e0 + j] - p[j] * through;
        }

        if (a.d_losses != nullptr) {
            const int s = find_seq(a.seq_offsets, a.num_seqs, static_cast<int>(t), lane);
            const int n = s >= 0 ? __ldg(a.seq_tokens + s) : 0;
            if (n > 0) {
                const float nf = static_cast<float>(n);
                const float gb = __ldg(a.d_losses + 2 * s) * (static_cast<float>(E) / (static_cast<float>(K) * nf)) / nf;
                const float gz = __ldg(a.d_losses + 2 * s + 1) * 2.0f * (m + logf(z)) / nf;
                const int32_t* cnt = a.counts + static_cast<int64_t>(s) * E + r.e0;
                float c[NPL], q[NPL];
#pragma unroll
                for (int j = 0; j < NPL; ++j)
                    c[j] = j < r.n ? static_cast<float>(__ldg(cnt + j)) : 0.0f;
                if (softmax || m < kSigmoidTail) {
#pragma unroll
                    for (int j = 0; j < NPL; ++j)
                        q[j] = p[j];
                } else {
                    float total = 0.0f;
#pragma unroll
                    for (int j = 0; j < NPL; ++j) {
                        q[j] = v[j] > kNegInf ? sigmoid(v[j]) : 0.0f;
                        total += q[j];
                    }
                    const float inv = 1.0f / warp_sum(total);
#pragma unroll
                    for (int j = 0; j < NPL; ++j)
                        q[j] *= inv;
                }
                float mean = 0.0f;
#pragma unroll
                for (int j = 0; j < NPL; ++j)
                    mean += c[j] * q[j];
                mean = warp_sum(mean);
#pragma unroll
                for (int j = 0; j < NPL; ++j) {
                    const float rest = softmax ? 1.0f : 1.0f / (1.0f + expf(v[j])); // ds/dl = s (1 - s)
                    d[j] += gb * q[j] * rest * (c[j] - mean) + gz * p[j];
                }
            }
        }
    }
    const int64_t at = t * E + r.e0;
    if (BF16) {
        uint16_t* out = static_cast<uint16_t*>(a.d_logits) + at;
        if (vec && NPL % 8 == 0) {
#pragma unroll
            for (int j = 0; j < NPL / 8; ++j)
                st_v4(out + 8 * j, make_uint4(pack_bf16x2(d[8 * j], d[8 * j + 1]), pack_bf16x2(d[8 * j + 2], d[8 * j + 3]),
                                              pack_bf16x2(d[8 * j + 4], d[8 * j + 5]),
                                              pack_bf16x2(d[8 * j + 6], d[8 * j + 7])));
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j < r.n)
                    out[j] = static_cast<uint16_t>(pack_bf16x2(d[j], 0.0f));
        }
    } else {
        float* out = static_cast<float*>(a.d_logits) + at;
        if (vec && NPL % 4 == 0) {
#pragma unroll
            for (int j = 0; j < NPL / 4; ++j)
                st_v4(out + 4 * j, make_uint4(__float_as_uint(d[4 * j]), __float_as_uint(d[4 * j + 1]),
                                              __float_as_uint(d[4 * j + 2]), __float_as_uint(d[4 * j + 3])));
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j < r.n)
                    out[j] = d[j];
        }
    }
}

// ----------------------------------------------------------------- launches
// Calls f<NPL, BF16>(vec) for the smallest NPL that holds a lane's run of
// logits.  vec: every lane has NPL logits and every run starts on 16 bytes.
template <typename F>
cudaError_t with_row_shape(const ep_router_desc_t& r, int groups, const void* in, const void* out, F&& f)
{
    const int c = run_length(r.num_experts, groups);
    const bool bf16 = r.logits_dtype == EP_BF16;
    const int size = bf16 ? 2 : 4;
    const bool vec = r.num_experts == 32 * c && (c * size) % 16 == 0 &&
                     ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
#define EP_ROW_SHAPE(N)                                                                                               \
    if (c <= N)                                                                                                       \
        return bf16 ? f(std::integral_constant<int, N>{}, std::true_type{}, vec && c == N)                            \
                    : f(std::integral_constant<int, N>{}, std::false_type{}, vec && c == N)
    EP_ROW_SHAPE(1);
    EP_ROW_SHAPE(2);
    EP_ROW_SHAPE(4);
    EP_ROW_SHAPE(8);
    EP_ROW_SHAPE(16);
    EP_ROW_SHAPE(32);
#undef EP_ROW_SHAPE
    return cudaErrorInvalidValue;
}

} // namespace

cudaError_t launch_router_topk(const RouterTopkLaunch& a, cudaStream_t stream)
{
    if (a.r.num_tokens == 0)
        return cudaSuccess;
    return with_row_shape(a.r, a.r.num_groups, a.logits, nullptr, [&](auto npl, auto bf16, bool vec) {
        const bool wide = a.bias != nullptr || a.r.num_groups > 1;
        const size_t smem = wide ? sizeof(double) * kTopkWarps * a.r.num_experts : 0;
        const unsigned grid = (a.r.num_tokens + kTopkWarps - 1) / kTopkWarps;
        router_topk_kernel<npl(), bf16()><<<grid, kTopkWarps * 32, smem, stream>>>(a, vec);
        return cudaGetLastError();
    });
}

size_t balance_workspace_bytes(int64_t T, int64_t E, int64_t S)
{
    const size_t bytes = static_cast<size_t>(balance_items(T, S)) * (8 * E + 8);
    return (bytes + 255) / 256 * 256;
}

cudaError_t launch_balance_loss(const BalanceLaunch& a, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (a.r.num_tokens > 0) {
        e = with_row_shape(a.r, 1, a.logits, nullptr, [&](auto npl, auto bf16, bool vec) {
            const size_t smem = sizeof(float) * (kBalanceWarps + 1) * a.r.num_experts;
            const unsigned grid = static_cast<unsigned>(balance_items(a.r.num_tokens, a.num_seqs));
            balance_chunk_kernel<npl(), bf16()><<<grid, kBalanceWarps * 32, smem, stream>>>(a, vec);
            return cudaGetLastError();
        });
    }
    if (e != cudaSuccess)
        return e;
    balance_finish_kernel<<<a.num_seqs, kFinishThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_router_backward(const RouterBackwardLaunch& a, cudaStream_t stream)
{
    if (a.r.num_tokens == 0)
        return cudaSuccess;
    return with_row_shape(a.r, 1, a.logits, a.d_logits, [&](auto npl, auto bf16, bool vec) {
        const size_t smem = sizeof(float) * kBackwardWarps * a.r.num_experts;
        const unsigned grid = (a.r.num_tokens + kBackwardWarps - 1) / kBackwardWarps;
        router_backward_kernel<npl(), bf16()><<<grid, kBackwardWarps * 32, smem, stream>>>(a, vec);
        return cudaGetLastError();
    });
}

} // namespace ep
