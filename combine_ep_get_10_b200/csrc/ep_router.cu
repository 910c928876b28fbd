// ep_router.cu -- the token router, its balance losses and their gradient.
//
// All kernels give a token's row of E <= 1024 logits to one warp and keep it in
// registers, NPL of them a lane (RowMap).  None is bound by its bytes at the sizes
// of a step (4096 x 256 logits are 0.6 us of memory): it is chains of dependent
// instructions, 10 cycles each, that last, so in the losses and the gradient the next
// row is on its way while one is worked on (the choice has one row a warp), and what
// few rows need (fp64) is kept short.
#include <algorithm>
#include <cfloat>

#include <cooperative_groups.h>

#include "ep_device.cuh"
#include "ep_router_launch.h"

namespace ep {

namespace cg = cooperative_groups;

namespace {

constexpr int kTopkWarps = 4;
constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------------ rows
// Which experts a lane's NPL registers hold.
//   without groups: vectors of kFull consecutive experts, vector after vector
//     dealt to the lanes (VEC, one 16-byte load each), or single ones where E or
//     the rows' alignment rules that out;
//   with groups: 32 / G lanes hold a group, `c` consecutive experts each, so
//     that a group is a run of whole lanes (VEC: c whole vectors).
template <int NPL, bool BF16, bool GROUPED, bool VEC>
struct RowMap {
    static constexpr int kFull = BF16 ? 8 : 4;
    int e0, n, E;

    __device__ __forceinline__ RowMap(const ep_router_desc_t& r, int lane) : E(r.num_experts)
    {
        if (GROUPED) {
            const int bits = 5 - (31 - __clz(r.num_groups)); // 2^bits lanes a group
            const int per = E >> (5 - bits), c = (per + (1 << bits) - 1) >> bits;
            const int q = lane & ((1 << bits) - 1);
            e0 = (lane >> bits) * per + min(q * c, per);
            n = max(0, min(c, per - q * c));
        } else {
            e0 = VEC ? lane * kFull : lane;
            n = E - e0;
        }
    }
    // Register j holds expert e0 + offset(j), if holds(j).
    static __device__ __forceinline__ constexpr int offset(int j)
    {
        return GROUPED ? j : (VEC ? (j / kFull) * (32 * kFull) + j % kFull : 32 * j);
    }
    __device__ __forceinline__ bool holds(int j) const { return offset(j) < n; }
};

int groups_run(const ep_router_desc_t& r) // c of RowMap
{
    const int lanes = 32 / r.num_groups;
    return (r.num_experts / r.num_groups + lanes - 1) / lanes;
}

// A logit as the operators take it: NaN closes the expert like -inf, values
// above the largest finite one count as that one (so that l - max is never
// inf - inf).
__device__ __forceinline__ float clean_logit(float l)
{
    return fminf(fmaxf(l, kNegInf), FLT_MAX); // fmaxf(NaN, x) is x
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i)
{
    if (BF16)
        return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(logits) + i)) << 16);
    return __ldg(static_cast<const float*>(logits) + i);
}

// Loads that are not waited for before their value is used: predicated, into
// the register that holds the value otherwise.  (A load in a branch is copied at
// the branch's end, and the copy, like any use, waits for it.)
__device__ __forceinline__ void load_u8_if(uint32_t& r, const uint8_t* p, bool on)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u8 %0, [%1];\n\t}"
                 : "+r"(r)
                 : "l"(p), "r"(on ? 1u : 0u));
}

__device__ __forceinline__ void load_u16_if(uint32_t& r, const void* p, bool on)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
                 : "+r"(r)
                 : "l"(p), "r"(on ? 1u : 0u));
}

__device__ __forceinline__ void load_u32_if(uint32_t& r, const void* p, bool on)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                 : "+r"(r)
                 : "l"(p), "r"(on ? 1u : 0u));
}

__device__ __forceinline__ void load_s64_if(int64_t& r, const int64_t* p, bool on)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.s64 %0, [%1];\n\t}"
                 : "+l"(r)
                 : "l"(p), "r"(on ? 1u : 0u));
}

// A lane's part of a row as it lies in memory, so that the next row can be on
// its way while one is worked on.
template <int NPL, bool BF16, bool GROUPED, bool VEC>
struct RawRow {
    using Map = RowMap<NPL, BF16, GROUPED, VEC>;
    static constexpr int kWords = VEC ? NPL * (BF16 ? 2 : 4) / 16 : NPL;
    uint4 vec[VEC ? kWords : 1];
    uint32_t one[VEC ? 1 : NPL];

    __device__ __forceinline__ void load(const void* logits, int64_t row, const Map& map, bool on)
    {
        const int64_t at = row * map.E + map.e0;
        if (VEC) {
            const uint32_t closed = BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
            for (int j = 0; j < NPL; j += Map::kFull) {
                uint4& w = vec[j / Map::kFull];
                w = make_uint4(closed, closed, closed, closed);
                const void* from = BF16 ? static_cast<const void*>(static_cast<const uint16_t*>(logits) + at + Map::offset(j))
                                        : static_cast<const void*>(static_cast<const float*>(logits) + at + Map::offset(j));
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                             "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                             : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)
                             : "l"(from), "r"(on && map.holds(j) ? 1u : 0u));
            }
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                one[j] = BF16 ? 0xff80u : 0xff800000u; // -inf
                if (BF16)
                    load_u16_if(one[j], static_cast<const uint16_t*>(logits) + at + Map::offset(j), on && map.holds(j));
                else
                    load_u32_if(one[j], static_cast<const float*>(logits) + at + Map::offset(j), on && map.holds(j));
            }
        }
    }
    // The logits, closed ones and registers that hold nothing as -inf.
    __device__ __forceinline__ void take(float (&v)[NPL]) const
    {
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            float l;
            if (VEC) {
                const uint4& w = vec[j / Map::kFull];
                const int i = j % Map::kFull, k = BF16 ? i / 2 : i;
                const uint32_t u = k == 0 ? w.x : (k == 1 ? w.y : (k == 2 ? w.z : w.w));
                l = BF16 ? (i % 2 == 0 ? bf16_lo(u) : bf16_hi(u)) : __uint_as_float(u);
            } else {
                l = __uint_as_float(BF16 ? one[j] << 16 : one[j]);
            }
            v[j] = clean_logit(l);
        }
    }
};

__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
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

// exp and sigmoid for whole rows: ex2.approx of l * log2(e) (2 ulp, and the
// product's half ulp, |l| * 2^-24 of the result) and a 2-ulp quotient.
__device__ __forceinline__ float fast_sigmoid(float l)
{
    return __fdividef(1.0f, 1.0f + __expf(-l));
}

// Below this, sigmoid(l) = exp(l) to fp32 precision, and ratios of sigmoids are
// taken as ratios of exponentials, which do not underflow.
constexpr float kSigmoidTail = -60.0f;

// -------------------------------------------------------------- selection
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

// Does the lane's group stay in the choice: in fp64, for the rows whose groups'
// fp32 values lie too close together.
template <int NPL, bool BF16, bool VEC>
__device__ __noinline__ bool stays_wide(const RouterTopkLaunch& a, int64_t row, int lane)
{
    const RowMap<NPL, BF16, true, VEC> map(a.r, lane);
    const int G = a.r.num_groups, bits = 5 - (31 - __clz(G));
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const double none = -INFINITY;
    RawRow<NPL, BF16, true, VEC> raw;
    float v[NPL];
    raw.load(a.logits, row, map, true);
    raw.take(v);
    double m = 0.0, z = 1.0;
    if (softmax) {
        m = fmaxf(row_max(v), -FLT_MAX);
        z = 0.0;
#pragma unroll 4
        for (int j = 0; j < NPL; ++j)
            z += exp(v[j] - m);
        for (int d = 16; d >= 1; d >>= 1)
            z += __shfl_xor_sync(kFullMask, z, d);
    }
    double t1 = none, t2 = none;
#pragma unroll 4
    for (int j = 0; j < NPL; ++j) {
        double c = softmax ? exp(v[j] - m) / z : 1.0 / (1.0 + exp(-static_cast<double>(v[j])));
        if (a.bias != nullptr && map.holds(j))
            c += __ldg(a.bias + map.e0 + map.offset(j));
        c = v[j] > kNegInf && c > none ? c : none;
        t2 = fmax(t2, fmin(t1, c));
        t1 = fmax(t1, c);
    }
    for (int d = (1 << bits) >> 1; d >= 1; d >>= 1) {
        const double o1 = __shfl_xor_sync(kFullMask, t1, d), o2 = __shfl_xor_sync(kFullMask, t2, d);
        t2 = fmax(fmin(t1, o1), fmax(t2, o2));
        t1 = fmax(t1, o1);
    }
    const double value = a.r.group_top == 2 && t2 > none ? t1 + t2 : t1;
    int before = 0;
    for (int g = 0; g < G; ++g) {
        const double o = __shfl_sync(kFullMask, value, g << bits);
        before += (o > value || (o == value && g < lane >> bits)) ? 1 : 0;
    }
    return before < a.r.topk_groups;
}

// Lane i of the first `count` gives its value and id: the lane's place in
// descending order, equal values by id.
template <typename T>
__device__ __forceinline__ int place_in_order(T value, int e, int count)
{
    int place = 0;
    for (int i = 0; i < count; ++i) {
        const T o = __shfl_sync(kFullMask, value, i);
        const int oe = __shfl_sync(kFullMask, e, i);
        place += (o > value || (o == value && oe < e)) ? 1 : 0;
    }
    return place;
}

// One warp a token: 128 x 256 fp32 2.5 us, 4096 x 256 in 8 groups with a bias 8.6
// us, 16381 x 160 bf16 9.6 us (0.55 TB/s), launches included.
//
// Selection.  Let t be the K-th largest of the 32 lanes' largest values: K
// values are at least t, so the K largest are among the values >= t, about a
// dozen for K = 8 of 256.  They are gathered to one a lane and put in order by
// counting, for each, those before it.  (If they are more than 32 - many equal
// values, or K near 32 - the K largest are taken one by one instead.)
//
// Order.  Without bias and groups the choice is by the logits themselves and
// exact.  Otherwise the fp32 values c carry an error of at most err(c): half
// an ulp of the sum with the bias (twice, for the comparison's own rounding), and
// that of s,
//   sigmoid: 2 ulp of ex2 and |l| * 2^-24 on s (1 - s) <= 1/4 and |l| s (1 - s)
//            <= 0.23, then the sum and the 2-ulp quotient: < 8 * 2^-24 < 5e-7;
//   softmax: on p <= 1 / Z, l - max and its product with log2(e) half an ulp each
//            (|l - max| exp(l - max) <= 0.37), 2 ulp of ex2, the sum of E terms
//            NPL + 5 roundings and the same errors inside (the mean of |l -
//            max| under p is at most log E <= 7), the quotient: < 64 * 2^-24 / Z;
// a row whose order those errors could change is decided in fp64: the groups,
// the gathered values alone where only their order is open, or (a value below t
// could come in) the whole row.  Such rows are few and slow, and a kernel lasts
// as long as its slowest row: at 4096 x 256 in 8 groups 10.5 us where every such
// row is done whole.  Values that are equal because logit and bias are equal
// need no second look.
// (The fp64 parts take registers: in groups 12 to 40 bytes a thread spill around
// them.)
enum class Choice { kLogit, kScore, kGrouped }; // by the logits, by scores, by scores in groups

template <int NPL, bool BF16, Choice CHOICE, bool VEC>
__global__ void __launch_bounds__(kTopkWarps * 32) router_topk_kernel(RouterTopkLaunch a)
{
    constexpr bool GROUPED = CHOICE == Choice::kGrouped, by_logit = CHOICE == Choice::kLogit;
    extern __shared__ double s_wide[];
    __shared__ float2 s_list[kTopkWarps][2][32]; // (value, expert): as gathered, in order
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + warp;
    const int E = a.r.num_experts, K = a.r.num_topk;
    const RowMap<NPL, BF16, GROUPED, VEC> map(a.r, lane);
    pdl_wait();
    if (t >= a.r.num_tokens)
        return;
    int64_t* idx_out = a.topk_idx + t * K;
    float* w_out = a.topk_weights + t * K;
    RawRow<NPL, BF16, GROUPED, VEC> raw;
    raw.load(a.logits, t, map, true);
    if (a.token_mask != nullptr && __ldg(a.token_mask + t) == 0) {
        if (lane < K) {
            idx_out[lane] = -1;
            w_out[lane] = 0.0f;
        }
        return;
    }
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    float c[NPL]; // the values chosen by; -inf: not to be chosen
    raw.take(c);

    float m = 0.0f, z = 1.0f;
    if (softmax && (!by_logit || a.r.normalize == 0)) {
        m = fmaxf(row_max(c), -FLT_MAX);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            sum += __expf(c[j] - m); // 0 for -inf
        z = warp_sum(sum);
    }
    const float es = softmax ? 4e-6f / z : 5e-7f;
    const auto err = [es](float x) { return es + 1.3e-7f * fabsf(x); };
    if (!by_logit) {
        const float inv_z = 1.0f / z;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            float s = softmax ? __expf(c[j] - m) * inv_z : fast_sigmoid(c[j]);
            if (a.bias != nullptr && map.holds(j))
                s += __ldg(a.bias + map.e0 + map.offset(j));
            c[j] = c[j] > kNegInf ? fmaxf(s, kNegInf) : kNegInf; // (a bias of NaN closes too)
        }
        if (GROUPED && a.r.topk_groups < a.r.num_groups) {
            const int G = a.r.num_groups, bits = 5 - (31 - __clz(G)), mine = lane >> bits;
            float t1 = kNegInf, t2 = kNegInf;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                t2 = fmaxf(t2, fminf(t1, c[j]));
                t1 = fmaxf(t1, c[j]);
            }
            for (int d = (1 << bits) >> 1; d >= 1; d >>= 1) {
                const float o1 = __shfl_xor_sync(kFullMask, t1, d), o2 = __shfl_xor_sync(kFullMask, t2, d);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            const bool two = a.r.group_top == 2 && t2 > kNegInf;
            const float value = two ? t1 + t2 : t1;
            const float ge = err(t1) + (two ? err(t2) : 0.0f) + 1.3e-7f * fabsf(value);
            int before = 0;
            for (int g = 0; g < G; ++g) {
                const float o = __shfl_sync(kFullMask, value, g << bits);
                before += (o > value || (o == value && g < mine)) ? 1 : 0;
            }
            bool stay = before < a.r.topk_groups;
            const float low = warp_min(stay ? value - ge : INFINITY);
            const float high = warp_max(stay || value == kNegInf ? kNegInf : value + ge);
            if (high > kNegInf && low <= high) // a group's place is open
                stay = stays_wide<NPL, BF16, VEC>(a, t, lane);
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                c[j] = stay ? c[j] : kNegInf;
        }
    }

    // lane k: the k-th chosen, and those after it as far as they are known
    int my_idx = -1;
    float my_c = kNegInf;
    float best = c[0];
#pragma unroll
    for (int j = 1; j < NPL; ++j)
        best = fmaxf(best, c[j]);
    // (two values more where the order has to be checked: what comes after the
    // K-th is then known, and what is not gathered is well below it)
    float least = kNegInf;
    const int values = by_logit ? K : K + 2;
    for (int k = 0; k < values; ++k) {
        least = warp_max(best);
        if (least == kNegInf)
            break;
        if (best == least)
            best = kNegInf;
    }
    const bool all = least == kNegInf; // everything that can be chosen is gathered
    least = fmaxf(least, -FLT_MAX);
    int count = 0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const bool in = c[j] >= least;
        const uint32_t who = __ballot_sync(kFullMask, in);
        const int at = count + __popc(who & ((1u << lane) - 1u));
        if (in && at < 32)
            s_list[warp][0][at] = make_float2(c[j], __int_as_float(map.e0 + map.offset(j)));
        count += __popc(who);
    }
    __syncwarp();
    float after = kNegInf; // one by one: the (K + 1)-th value
    if (count <= 32) {
        float2 mine = make_float2(kNegInf, 0.0f);
        if (lane < count)
            mine = s_list[warp][0][lane];
        const int id = __float_as_int(mine.y);
        int place = 0;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float2 o = s_list[warp][0][i];
            place += (o.x > mine.x || (o.x == mine.x && __float_as_int(o.y) < id)) ? 1 : 0;
        }
        if (lane < count)
            s_list[warp][1][place] = mine;
        __syncwarp();
        if (lane < count) {
            mine = s_list[warp][1][lane];
            my_c = mine.x;
            my_idx = __float_as_int(mine.y);
        }
    } else {
        for (int k = 0; k <= K; ++k) {
            float top = kNegInf;
            int e = E;
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (c[j] > top) {
                    top = c[j];
                    e = map.e0 + map.offset(j);
                }
            after = warp_max(top);
            if (after == kNegInf)
                break;
            const int first = static_cast<int>(__reduce_min_sync(kFullMask, static_cast<uint32_t>(top == after ? e : E)));
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (map.e0 + map.offset(j) == first)
                    c[j] = kNegInf;
            if (lane == k && k < K) {
                my_idx = first;
                my_c = after;
            }
        }
    }
    float l = my_c; // the logit itself without bias and groups
    if (!by_logit) {
        l = my_idx >= 0 ? clean_logit(load_logit<BF16>(a.logits, t * E + my_idx)) : 0.0f;
        const float b = my_idx >= 0 && a.bias != nullptr ? __ldg(a.bias + my_idx) : 0.0f;
        float n = __shfl_down_sync(kFullMask, my_c, 1);
        const float nl = __shfl_down_sync(kFullMask, l, 1), nb = __shfl_down_sync(kFullMask, b, 1);
        const float last = __shfl_sync(kFullMask, my_c, K - 1); // -inf: fewer than K
        // the order of the chosen, and of what is equal to the last of them
        bool like = l == nl && b == nb;
        const bool open = lane < K || my_c == last;
        if (lane == 31)
            n = kNegInf;
        if (count > 32 && lane == K - 1) {
            n = after; // more of these values may follow: equal ones settle nothing
            like = false;
        }
        const bool order = __all_sync(kFullMask, !open || my_c == kNegInf || n == kNegInf || like ||
                                                     my_c - err(my_c) > n + err(n));
        // what was not gathered is below `least`
        const bool closed = all || count > 32 || last - err(last) > least + err(least);
        if (!closed || (!order && count > 32)) {
            my_idx = choose_wide<BF16>(a, t, s_wide + static_cast<size_t>(warp) * E, lane);
            l = my_idx >= 0 ? clean_logit(load_logit<BF16>(a.logits, t * E + my_idx)) : 0.0f;
        } else if (!order) {
            double sum = 1.0;
            if (softmax) {
                sum = 0.0;
#pragma unroll 4
                for (int e = lane; e < E; e += 32)
                    sum += exp(static_cast<double>(clean_logit(load_logit<BF16>(a.logits, t * E + e))) - m);
                for (int d = 16; d >= 1; d >>= 1)
                    sum += __shfl_xor_sync(kFullMask, sum, d);
            }
            const double l64 = l;
            const double c64 = (softmax ? exp(l64 - m) / sum : 1.0 / (1.0 + exp(-l64))) + b;
            const int place = place_in_order(c64, my_idx, count);
            if (lane < count)
                s_list[warp][0][place] = make_float2(l, __int_as_float(my_idx));
            __syncwarp();
            if (lane < count) {
                l = s_list[warp][0][lane].x;
                my_idx = __float_as_int(s_list[warp][0][lane].y);
            }
        }
    }
    if (lane >= K)
        my_idx = -1;

    const bool got = my_idx >= 0;
    float w = 0.0f;
    if (a.r.normalize != 0) {
        const float lm = warp_max(got ? l : kNegInf);
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
// Tokens are dealt out in chunks of at most `chunk` tokens of one sequence,
// sequence after sequence.  A CTA sums a chunk; where that is the whole
// sequence it writes the results, else it leaves its sums in the workspace and
// a cluster of the second kernel adds the sequence's up in a fixed order (fixed
// order, no floating-point atomics, nothing that one call leaves for the next).
constexpr int kBalanceWarps = 16;
constexpr int kBalanceThreads = kBalanceWarps * 32;
// Chunks of a long batch, one an SM: at 4096 x 256 14.4 us a loss and gradient, with
// two an SM 16.3 us; at 16384 x 256 in 13 sequences 24.5 and 22.1 us.
constexpr int kBalanceCtas = 148;
constexpr int kFewTokens = 256; // one chunk a sequence: 128 x 8 3 us less of a caller's time

// Tokens a chunk, a multiple of the warps.  Few tokens make one chunk each
// sequence: the second launch would cost more than the longer sums.
int chunk_tokens(int64_t T)
{
    const int64_t each = T <= kFewTokens ? T : (T + kBalanceCtas - 1) / kBalanceCtas;
    return static_cast<int>((each + kBalanceWarps - 1) / kBalanceWarps * kBalanceWarps);
}

// The chunks of sequence s are numbered from begin / chunk + s on: a sequence of n
// tokens has at most n / chunk + 1 of them, so numbers do not meet, some stay
// unused, and a number's sequence is found by bisection, a sequence's numbers
// without a look at the others.  T / chunk + S are enough, which is at most this; it
// grows with T.
__host__ __device__ __forceinline__ int64_t most_chunks(int64_t T, int64_t S)
{
    const int64_t full = (T + kBalanceWarps - 1) / kBalanceWarps;
    return (full < kBalanceCtas ? full : kBalanceCtas) + S;
}

// Workspace: each chunk's sums (score, count) per expert, then its (sum of
// lse^2, tokens).
struct BalanceSums {
    int2* sums;  // [chunks, E]: bits of the fp32 sum, count
    int2* tails; // [chunks]: bits of the fp32 sum, tokens
};

__device__ __forceinline__ BalanceSums balance_sums(void* workspace, int64_t chunks, int E)
{
    int2* sums = static_cast<int2*>(workspace);
    return {sums, sums + chunks * E};
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

// How many of the `count` values f(0) <= f(1) <= .. are at most x: each step reads 32
// of them spread over what is left.  One warp; lanes agree.  (Whatever f gives, the
// answer is in [0, count].)
template <typename F>
__device__ __forceinline__ int count_up_to(int count, int x, int lane, F&& f)
{
    int lo = 0, len = count; // lo of them so far
    while (len > 0) {
        const int step = (len + 31) / 32;
        const int at = lo + (lane + 1) * step - 1; // the last one of the lane's run
        const bool le = at < lo + len && f(at) <= x;
        const int runs = __popc(__ballot_sync(kFullMask, le));
        lo += runs * step;
        if (step == 1)
            break;
        len = min(step - 1, count - lo);
    }
    return lo;
}

// The sequence of token t (the last one that begins at or before it), -1 when
// it is in none.
__device__ __forceinline__ int find_seq(const int32_t* offsets, int S, int t, int lane)
{
    if (offsets == nullptr)
        return 0;
    const int s = count_up_to(S + 1, t, lane, [&](int i) { return __ldg(offsets + i); }) - 1;
    return s < S ? s : -1;
}

struct Chunk {
    int seq, of; // the sequence, its number of chunks
    TokenRange tokens;
};

// A sequence's first chunk, and how many it has.
__device__ __forceinline__ int first_chunk(const TokenRange& r, int chunk, int s)
{
    return r.begin / chunk + s;
}

__device__ __forceinline__ int chunks_of(const TokenRange& r, int chunk)
{
    return (r.end - r.begin + chunk - 1) / chunk;
}

// Chunk i; `of` is 0 for a number that no sequence uses.  One warp; lanes agree.
__device__ __forceinline__ Chunk find_chunk(const int32_t* offsets, int T, int S, int chunk, int i, int lane)
{
    const int s = count_up_to(S, i, lane, [&](int j) { return first_chunk(seq_range(offsets, T, j), chunk, j); }) - 1;
    Chunk c{};
    if (s < 0)
        return c;
    const TokenRange r = seq_range(offsets, T, s);
    const int at = i - first_chunk(r, chunk, s), of = chunks_of(r, chunk);
    if (at < 0 || at >= of)
        return c;
    c.seq = s;
    c.of = of;
    c.tokens.begin = r.begin + at * chunk;
    c.tokens.end = min(r.end, c.tokens.begin + chunk);
    return c;
}

// The results of sequence s from its sums: thread e < E holds expert e's.  All
// threads of the CTA; red: kBalanceWarps floats of shared memory.
__device__ __forceinline__ void write_balance(const BalanceLaunch& a, int s, int tokens, float lse2, const float* q,
                                              const int* cnt, float* red)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.r.num_experts;
    const float n = static_cast<float>(tokens);
    float fp = 0.0f;
    for (int e = tid; e < E; e += kBalanceThreads) {
        const float mean = tokens > 0 ? q[e] / n : 0.0f;
        const int64_t at = static_cast<int64_t>(s) * E + e;
        a.counts[at] = tokens > 0 ? cnt[e] : 0;
        if (a.mean_scores != nullptr)
            a.mean_scores[at] = mean;
        fp += static_cast<float>(cnt[e]) * mean;
    }
    fp = warp_sum(fp);
    if (lane == 0)
        red[warp] = fp;
    __syncthreads();
    if (tid == 0) {
        float sum = 0.0f;
        for (int w = 0; w < kBalanceWarps; ++w)
            sum += red[w];
        const float scale = static_cast<float>(E) / (static_cast<float>(a.r.num_topk) * n);
        a.losses[2 * s] = tokens > 0 ? sum * scale : 0.0f;
        a.losses[2 * s + 1] = tokens > 0 ? lse2 / n : 0.0f;
        a.seq_tokens[s] = tokens;
    }
}

template <int NPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(kBalanceThreads) balance_kernel(BalanceLaunch a, int chunk, bool finish)
{
    extern __shared__ float s_q[]; // [kBalanceWarps, E] each warp's sums, [E] the experts' counts
    __shared__ float s_z[kBalanceWarps], s_red[kBalanceWarps];
    __shared__ int s_n[kBalanceWarps];
    __shared__ Chunk s_chunk;
    pdl_wait();
    if (finish)
        pdl_launch_dependents(); // balance_finish_kernel, which waits for this grid
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.r.num_experts, K = a.r.num_topk, T = a.r.num_tokens, S = a.num_seqs;
    int* s_cnt = reinterpret_cast<int*>(s_q + kBalanceWarps * E);
    const int64_t chunks = most_chunks(T, S);
    const BalanceSums part = balance_sums(a.workspace, chunks, E);
    if (warp == 0) {
        const Chunk found = find_chunk(a.seq_offsets, T, S, chunk, blockIdx.x, lane);
        if (lane == 0)
            s_chunk = found;
    }
    if (static_cast<int>(blockIdx.x) < S) { // a sequence without tokens
        const int64_t s = blockIdx.x;
        const TokenRange r = seq_range(a.seq_offsets, T, static_cast<int>(s));
        if (r.begin >= r.end) {
            for (int e = tid; e < E; e += kBalanceThreads) {
                a.counts[s * E + e] = 0;
                if (a.mean_scores != nullptr)
                    a.mean_scores[s * E + e] = 0.0f;
            }
            if (tid == 0) {
                a.losses[2 * s] = a.losses[2 * s + 1] = 0.0f;
                a.seq_tokens[s] = 0;
            }
        }
    }
    __syncthreads();
    const Chunk c = s_chunk;
    if (c.of == 0)
        return;
    for (int e = tid; e < E; e += kBalanceThreads)
        s_cnt[e] = 0;
    __syncthreads();

    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const RowMap<NPL, BF16, false, VEC> map(a.r, lane);
    float acc[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        acc[j] = 0.0f;
    float zz = 0.0f;
    int live = 0;
    // one token a warp: its row, mask and ids are loaded while the one before is summed
    RawRow<NPL, BF16, false, VEC> raw;
    int64_t e_next;
    uint32_t mask_next;
    const auto load = [&](int t) {
        const bool in = t < c.tokens.end;
        raw.load(a.logits, t, map, in);
        mask_next = 1u;
        load_u8_if(mask_next, a.token_mask + t, in && a.token_mask != nullptr);
        e_next = -1;
        load_s64_if(e_next, a.topk_idx + static_cast<int64_t>(t) * K + lane, in && lane < K);
    };
    load(c.tokens.begin + warp);
    for (int t = c.tokens.begin + warp; t < c.tokens.end; t += kBalanceWarps) {
        float v[NPL];
        raw.take(v);
        const int64_t e = e_next;
        const bool on = mask_next != 0u;
        load(t + kBalanceWarps);
        if (!on)
            continue;
        const float m = row_max(v);
        if (!(m > kNegInf))
            continue; // every expert closed
        if (e >= 0 && e < E)
            atomicAdd(s_cnt + e, 1);
        ++live;
        float sum = 0.0f;
        float p[NPL];
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            p[j] = __expf(v[j] - m); // 0 for -inf
            sum += p[j];
        }
        sum = warp_sum(sum);
        const float lse = m + logf(sum);
        zz += lse * lse;
        if (!softmax && m >= kSigmoidTail) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                p[j] = v[j] > kNegInf ? fast_sigmoid(v[j]) : 0.0f;
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
        if (map.holds(j))
            s_q[warp * E + map.e0 + map.offset(j)] = acc[j];
    if (lane == 0) {
        s_z[warp] = zz;
        s_n[warp] = live;
    }
    __syncthreads();
    for (int e = tid; e < E; e += kBalanceThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalanceWarps; ++w)
            sum += s_q[w * E + e];
        s_q[e] = sum; // only this thread reads the column again
        if (c.of > 1)
            part.sums[static_cast<int64_t>(blockIdx.x) * E + e] = make_int2(__float_as_int(sum), s_cnt[e]);
    }
    float z = 0.0f;
    int n = 0;
    for (int w = 0; w < kBalanceWarps; ++w) {
        z += s_z[w];
        n += s_n[w];
    }
    if (c.of == 1) {
        write_balance(a, c.seq, n, z, s_q, s_cnt, s_red);
        return;
    }
    if (tid == 0)
        part.tails[blockIdx.x] = make_int2(__float_as_int(z), n);
}

// The results of the sequences that are made of several chunks, a cluster each.
// Where there are more sequences than chunks (by_token), cluster j takes the one that
// token j * chunk is the first such token of: those of several chunks all have one,
// and there are no more clusters than chunks, however many sequences.
// The CTAs share out the experts and, in each, the warps the chunks (one CTA
// alone would draw all the partial sums through one SM: 7 us for 148 chunks of
// 256 experts).
constexpr int kFinishCluster = 8;
constexpr int kFinishLoads = 10; // 16 warps: 160 chunks in one go, the most a sequence of a long batch has
constexpr int kFinishExperts = kRouterMaxExperts / kFinishCluster; // a CTA, at most

__global__ void __launch_bounds__(kBalanceThreads) balance_finish_kernel(BalanceLaunch a, int chunk, bool by_token)
{
    __shared__ float s_q[kBalanceWarps][kFinishExperts];
    __shared__ int s_cnt[kBalanceWarps][kFinishExperts];
    __shared__ float s_z, s_red[kBalanceWarps], s_sum;
    __shared__ int s_n;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = static_cast<int>(cluster.block_rank());
    const int E = a.r.num_experts, T = a.r.num_tokens, S = a.num_seqs, j = blockIdx.x / kFinishCluster;
    const int64_t chunks = most_chunks(T, S);
    const BalanceSums part = balance_sums(a.workspace, chunks, E);
    // (what it reads before the wait is older than the kernel that it waits for)
    const int s = by_token ? find_seq(a.seq_offsets, S, j * chunk, lane) : j;
    const TokenRange own = s >= 0 ? seq_range(a.seq_offsets, T, s) : TokenRange{0, 0};
    pdl_wait();
    const int64_t before = static_cast<int64_t>(j - 1) * chunk;
    if (own.end - own.begin <= chunk || (by_token && own.begin <= before))
        return; // one chunk at most, or another cluster's: the whole cluster
    const int first = first_chunk(own, chunk, s), of = chunks_of(own, chunk);
    const int per = (E + kFinishCluster - 1) / kFinishCluster, e0 = min(rank * per, E), n_e = min(per, E - e0);
    for (int x = lane; x < n_e; x += 32) {
        float q = 0.0f;
        int cnt = 0;
        for (int base = warp; base < of; base += kFinishLoads * kBalanceWarps) {
            int2 o[kFinishLoads]; // all on their way at once
#pragma unroll
            for (int u = 0; u < kFinishLoads; ++u) {
                const int i = base + u * kBalanceWarps;
                o[u] = i < of ? __ldcg(part.sums + static_cast<int64_t>(first + i) * E + e0 + x) : make_int2(0, 0);
            }
#pragma unroll
            for (int u = 0; u < kFinishLoads; ++u) {
                q += __int_as_float(o[u].x);
                cnt += o[u].y;
            }
        }
        s_q[warp][x] = q;
        s_cnt[warp][x] = cnt;
    }
    if (warp == kBalanceWarps - 1) { // every CTA needs the tokens
        float z = 0.0f;
        int n = 0;
        for (int base = lane; base < of; base += 5 * 32) {
            int2 o[5];
#pragma unroll
            for (int u = 0; u < 5; ++u)
                o[u] = base + 32 * u < of ? __ldcg(part.tails + first + base + 32 * u) : make_int2(0, 0);
#pragma unroll
            for (int u = 0; u < 5; ++u) {
                z += __int_as_float(o[u].x);
                n += o[u].y;
            }
        }
        z = warp_sum(z);
        n = __reduce_add_sync(kFullMask, n);
        if (lane == 0) {
            s_z = z;
            s_n = n;
        }
    }
    __syncthreads();
    const int tokens = s_n;
    const float nf = static_cast<float>(tokens);
    float fp = 0.0f;
    if (tid < n_e) {
        float q = 0.0f;
        int cnt = 0;
#pragma unroll
        for (int w = 0; w < kBalanceWarps; ++w) {
            q += s_q[w][tid];
            cnt += s_cnt[w][tid];
        }
        const float mean = tokens > 0 ? q / nf : 0.0f;
        const int64_t at = static_cast<int64_t>(s) * E + e0 + tid;
        a.counts[at] = tokens > 0 ? cnt : 0;
        if (a.mean_scores != nullptr)
            a.mean_scores[at] = mean;
        fp = static_cast<float>(cnt) * mean;
    }
    fp = warp_sum(fp);
    if (lane == 0)
        s_red[warp] = fp;
    __syncthreads();
    if (tid == 0) {
        float sum = 0.0f;
        for (int w = 0; w < kBalanceWarps; ++w)
            sum += s_red[w];
        s_sum = sum;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
        float sum = 0.0f;
        for (int i = 0; i < kFinishCluster; ++i)
            sum += *cluster.map_shared_rank(&s_sum, i);
        a.losses[2 * s] = tokens > 0 ? sum * (static_cast<float>(E) / (static_cast<float>(a.r.num_topk) * nf)) : 0.0f;
        a.losses[2 * s + 1] = tokens > 0 ? s_z / nf : 0.0f;
        a.seq_tokens[s] = tokens;
    }
    cluster.sync(); // no CTA leaves while its sum is read
}

// ---------------------------------------------------------------- backward
constexpr int kBackwardWarps = 4;
// Warps to keep before runs get longer: at 16384 x 256 24.5 us a loss and
// gradient, with 16 an SM 26.1 us, with 32 26.7 us.
constexpr int kBackwardFill = 148 * 24;
constexpr int kMostRun = 16;

// 16 bytes of shared or global memory at a time where the lane's experts lie
// together.
template <int NPL, bool BF16, bool VEC, typename F4, typename F1>
__device__ __forceinline__ void each_expert(const RowMap<NPL, BF16, false, VEC>& map, F4&& four, F1&& one)
{
    using Map = RowMap<NPL, BF16, false, VEC>;
    if (VEC) {
#pragma unroll
        for (int j = 0; j < NPL; j += 4)
            if (map.holds(j))
                four(j, map.e0 + Map::offset(j));
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (map.holds(j))
                one(j, map.e0 + Map::offset(j));
    }
}

// A warp has `run` consecutive tokens: the next one's row, mask, ids and
// gradients are on their way while one is worked on, and the counts of a
// sequence stay in registers until its last token.  Latencies bound it: 64
// registers, for 32 warps an SM, take 14.4 us for loss and gradient of 4096 x
// 256, 80 registers 15.7 us, though at 8 logits a lane (256 experts) 40 to 100 bytes a
// thread spill.
template <int NPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(kBackwardWarps * 32, NPL <= 8 ? 8 : 1) router_backward_kernel(RouterBackwardLaunch a, int run)
{
    extern __shared__ __align__(16) float s_add[]; // [kBackwardWarps, E]: the chosen experts' part
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.r.num_experts, K = a.r.num_topk;
    const bool softmax = a.r.score == EP_SCORE_SOFTMAX;
    const RowMap<NPL, BF16, false, VEC> map(a.r, lane);
    using Map = RowMap<NPL, BF16, false, VEC>;
    float* add = s_add + static_cast<size_t>(warp) * E;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kBackwardWarps + warp) * run;
    pdl_wait();
    if (first >= a.r.num_tokens)
        return;
    const int begin = static_cast<int>(first), end = static_cast<int>(min(first + run, static_cast<int64_t>(a.r.num_tokens)));
    RawRow<NPL, BF16, false, VEC> raw;
    int64_t e_next;
    uint32_t mask_next, g_next;
    const auto load = [&](int t) {
        const bool in = t < end, slot = in && a.d_topk_weights != nullptr && lane < K;
        const int64_t at = static_cast<int64_t>(t) * K + lane;
        raw.load(a.logits, t, map, in);
        mask_next = 1u;
        load_u8_if(mask_next, a.token_mask + t, in && a.token_mask != nullptr);
        e_next = -1;
        load_s64_if(e_next, a.topk_idx + at, slot);
        g_next = 0u;
        load_u32_if(g_next, a.d_topk_weights + at, slot);
    };
    load(begin);
    // the sequence at hand: its end, its losses' gradients over its tokens, its counts
    int seq_end = begin;
    float gb = 0.0f, gz = 0.0f, cnt[NPL];
    const auto enter = [&](int t) {
        const int s = find_seq(a.seq_offsets, a.num_seqs, t, lane);
        const int n = s >= 0 ? __ldg(a.seq_tokens + s) : 0;
        // (a sequence that does not hold t has no tokens here; look again at the next one)
        seq_end = a.seq_offsets == nullptr ? a.r.num_tokens : (s >= 0 ? max(__ldg(a.seq_offsets + s + 1), t + 1) : t + 1);
        gb = gz = 0.0f;
        if (s < 0)
            return;
        const float nf = static_cast<float>(max(n, 1)); // (no token of a sequence with n = 0 gets here)
        gb = __ldg(a.d_losses + 2 * s) * (static_cast<float>(E) / (static_cast<float>(K) * nf)) / nf;
        gz = __ldg(a.d_losses + 2 * s + 1) * 2.0f / nf;
        const int32_t* from = a.counts + static_cast<int64_t>(s) * E;
        each_expert<NPL, BF16, VEC>(
            map,
            [&](int j, int e) {
                const int4 c = __ldg(reinterpret_cast<const int4*>(from + e));
                cnt[j] = static_cast<float>(c.x);
                cnt[(j + 1) % NPL] = static_cast<float>(c.y);
                cnt[(j + 2) % NPL] = static_cast<float>(c.z);
                cnt[(j + 3) % NPL] = static_cast<float>(c.w);
            },
            [&](int j, int e) { cnt[j] = static_cast<float>(__ldg(from + e)); });
    };
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        cnt[j] = 0.0f;

    if (a.d_losses != nullptr)
        enter(begin);
    for (int t = begin; t < end; ++t) {
        float v[NPL], d[NPL];
        const int64_t e = e_next;
        float g = __uint_as_float(g_next);
        const bool on = mask_next != 0u;
        // lane k: slot k's logit
        uint32_t slot_l = BF16 ? 0xff80u : 0xff800000u;
        const bool slot = on && e >= 0 && e < E;
        if (BF16)
            load_u16_if(slot_l, static_cast<const uint16_t*>(a.logits) + static_cast<int64_t>(t) * E + e, slot);
        else
            load_u32_if(slot_l, static_cast<const float*>(a.logits) + static_cast<int64_t>(t) * E + e, slot);
        raw.take(v);
        load(t + 1);
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            d[j] = 0.0f;
        const float m = on ? row_max(v) : kNegInf;
        if (m > kNegInf) {
            // softmax of the row
            float p[NPL];
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                p[j] = __expf(v[j] - m); // 0 for -inf
                z += p[j];
            }
            z = warp_sum(z);
            const float inv_z = 1.0f / z;
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                p[j] *= inv_z;

            if (a.d_topk_weights != nullptr) {
                const float l = clean_logit(__uint_as_float(BF16 ? slot_l << 16 : slot_l));
                const bool got = l > kNegInf;
                g = got ? a.r.scale * g : 0.0f;
                float part = 0.0f;    // what slot k adds at its expert
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
                each_expert<NPL, BF16, VEC>(
                    map, [&](int, int x) { *reinterpret_cast<float4*>(add + x) = make_float4(0.0f, 0.0f, 0.0f, 0.0f); },
                    [&](int, int x) { add[x] = 0.0f; });
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
                each_expert<NPL, BF16, VEC>(
                    map,
                    [&](int j, int x) {
                        const float4 f = *reinterpret_cast<const float4*>(add + x);
                        d[j] = f.x;
                        d[(j + 1) % NPL] = f.y;
                        d[(j + 2) % NPL] = f.z;
                        d[(j + 3) % NPL] = f.w;
                    },
                    [&](int j, int x) { d[j] = add[x]; });
                __syncwarp(); // read before the next token's zeros
#pragma unroll
                for (int j = 0; j < NPL; ++j)
                    d[j] -= p[j] * through;
            }

            if (a.d_losses != nullptr) {
                if (t >= seq_end)
                    enter(t);
                const float gzt = gz * (m + logf(z));
                if (softmax || m < kSigmoidTail) { // there 1 - s is 1 too
                    float mean = 0.0f;
#pragma unroll
                    for (int j = 0; j < NPL; ++j)
                        mean += cnt[j] * p[j];
                    const float flat = gzt - gb * warp_sum(mean);
#pragma unroll
                    for (int j = 0; j < NPL; ++j)
                        d[j] += p[j] * (gb * cnt[j] + flat);
                } else {
                    float q[NPL];
                    float total = 0.0f;
#pragma unroll
                    for (int j = 0; j < NPL; ++j) {
                        q[j] = v[j] > kNegInf ? fast_sigmoid(v[j]) : 0.0f;
                        total += q[j];
                    }
                    const float inv = 1.0f / warp_sum(total);
                    float mean = 0.0f;
#pragma unroll
                    for (int j = 0; j < NPL; ++j) {
                        q[j] *= inv;
                        mean += cnt[j] * q[j];
                    }
                    mean = warp_sum(mean);
#pragma unroll
                    for (int j = 0; j < NPL; ++j) // 1 - s, kept exact where s is near 1
                        d[j] += gb * q[j] * fast_sigmoid(-v[j]) * (cnt[j] - mean) + gzt * p[j];
                }
            }
        }
        const int64_t at = static_cast<int64_t>(t) * E + map.e0;
        if (VEC) {
#pragma unroll
            for (int j = 0; j < NPL; j += Map::kFull) {
                if (!map.holds(j))
                    continue;
                uint4 w;
                if (BF16) {
                    w = make_uint4(pack_bf16x2(d[j], d[(j + 1) % NPL]), pack_bf16x2(d[(j + 2) % NPL], d[(j + 3) % NPL]),
                                   pack_bf16x2(d[(j + 4) % NPL], d[(j + 5) % NPL]),
                                   pack_bf16x2(d[(j + 6) % NPL], d[(j + 7) % NPL]));
                    st_v4(static_cast<uint16_t*>(a.d_logits) + at + Map::offset(j), w);
                } else {
                    w = make_uint4(__float_as_uint(d[j]), __float_as_uint(d[(j + 1) % NPL]),
                                   __float_as_uint(d[(j + 2) % NPL]), __float_as_uint(d[(j + 3) % NPL]));
                    st_v4(static_cast<float*>(a.d_logits) + at + Map::offset(j), w);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                if (!map.holds(j))
                    continue;
                if (BF16)
                    static_cast<uint16_t*>(a.d_logits)[at + Map::offset(j)] =
                        static_cast<uint16_t>(pack_bf16x2(d[j], 0.0f));
                else
                    static_cast<float*>(a.d_logits)[at + Map::offset(j)] = d[j];
            }
        }
    }
}

// ----------------------------------------------------------------- launches
// A launch as a programmatic dependent, in clusters of `cluster`: it is ready
// when the kernel before it ends, and every kernel here waits (pdl_wait) before
// it reads what that one may have written.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, int cluster,
                         cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Calls f<NPL, BF16, VEC> for the smallest NPL that holds a lane's logits; VEC:
// by 16-byte loads, where E is a multiple of that many logits and the arrays
// (`align`: their addresses, or'ed) start on 16 bytes.
template <typename F>
cudaError_t with_row_shape(const ep_router_desc_t& r, uintptr_t align, F&& f)
{
    const bool bf16 = r.logits_dtype == EP_BF16;
    const int full = bf16 ? 8 : 4;
    int need = (r.num_experts + 31) / 32;
    bool vec = (align & 15u) == 0 && r.num_experts % full == 0;
    if (r.num_groups > 1) { // runs of c, each of whole vectors
        need = groups_run(r);
        vec = vec && need >= full && (need & (need - 1)) == 0 && r.num_experts == 32 * need;
    } else if (vec) {
        need = (r.num_experts / full + 31) / 32 * full;
    }
#define EP_ROW_SHAPE(N)                                                                                               \
    if (need <= N) {                                                                                                  \
        using Npl = std::integral_constant<int, N>;                                                                   \
        if (bf16)                                                                                                     \
            return vec ? f(Npl{}, std::true_type{}, std::integral_constant<bool, (N >= 8)>{})                         \
                       : f(Npl{}, std::true_type{}, std::false_type{});                                               \
        return vec ? f(Npl{}, std::false_type{}, std::integral_constant<bool, (N >= 4)>{})                            \
                   : f(Npl{}, std::false_type{}, std::false_type{});                                                  \
    }
    EP_ROW_SHAPE(1);
    EP_ROW_SHAPE(2);
    EP_ROW_SHAPE(4);
    EP_ROW_SHAPE(8);
    EP_ROW_SHAPE(16);
    EP_ROW_SHAPE(32);
#undef EP_ROW_SHAPE
    return cudaErrorInvalidValue;
}

uintptr_t address(const void* p)
{
    return reinterpret_cast<uintptr_t>(p);
}

} // namespace

cudaError_t launch_router_topk(const RouterTopkLaunch& a, cudaStream_t stream)
{
    if (a.r.num_tokens == 0)
        return cudaSuccess;
    return with_row_shape(a.r, address(a.logits), [&](auto npl, auto bf16, auto vec) {
        const bool grouped = a.r.num_groups > 1;
        const size_t smem = grouped || a.bias != nullptr ? sizeof(double) * kTopkWarps * a.r.num_experts : 0;
        const unsigned grid = (a.r.num_tokens + kTopkWarps - 1) / kTopkWarps;
        return launch_after(grouped             ? router_topk_kernel<npl(), bf16(), Choice::kGrouped, vec()>
                            : a.bias != nullptr ? router_topk_kernel<npl(), bf16(), Choice::kScore, vec()>
                                                : router_topk_kernel<npl(), bf16(), Choice::kLogit, vec()>,
                            grid, kTopkWarps * 32, smem, 1, stream, a);
    });
}

size_t balance_workspace_bytes(int64_t T, int64_t E, int64_t S)
{
    const size_t bytes = static_cast<size_t>(most_chunks(T, S)) * (8 * E + 8);
    return (bytes + 255) / 256 * 256;
}

cudaError_t launch_balance_loss(const BalanceLaunch& a, cudaStream_t stream)
{
    ep_router_desc_t r = a.r;
    r.num_groups = 1; // the groups are the choice's alone
    return with_row_shape(r, address(a.logits), [&](auto npl, auto bf16, auto vec) {
        const auto kernel = balance_kernel<npl(), bf16(), vec()>;
        const size_t smem = sizeof(float) * (kBalanceWarps + 1) * a.r.num_experts;
        if (smem > 47 * 1024) { // 48 KB, the kernel's own arrays among them, need no leave
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess)
                return e;
        }
        const int T = a.r.num_tokens, chunk = chunk_tokens(std::max(T, 1));
        const unsigned grid = static_cast<unsigned>(T / chunk + a.num_seqs);
        const bool finish = T > chunk; // else no sequence has a second chunk
        const cudaError_t e = launch_after(kernel, grid, kBalanceThreads, smem, 1, stream, a, chunk, finish);
        if (e != cudaSuccess || !finish)
            return e;
        const int tokens = (T - 1) / chunk + 1;
        const bool by_token = a.num_seqs > tokens;
        return launch_after(balance_finish_kernel, static_cast<unsigned>(by_token ? tokens : a.num_seqs) * kFinishCluster,
                            kBalanceThreads, 0, kFinishCluster, stream, a, chunk, by_token);
    });
}

cudaError_t launch_router_backward(const RouterBackwardLaunch& a, cudaStream_t stream)
{
    if (a.r.num_tokens == 0)
        return cudaSuccess;
    ep_router_desc_t r = a.r;
    r.num_groups = 1;
    const uintptr_t align = address(a.logits) | address(a.d_logits) | (a.d_losses != nullptr ? address(a.counts) : 0);
    return with_row_shape(r, align, [&](auto npl, auto bf16, auto vec) {
        const size_t smem = sizeof(float) * kBackwardWarps * a.r.num_experts;
        const int run = std::max(1, std::min(kMostRun, a.r.num_tokens / kBackwardFill));
        const unsigned grid = (a.r.num_tokens + kBackwardWarps * run - 1) / (kBackwardWarps * run);
        return launch_after(router_backward_kernel<npl(), bf16(), vec()>, grid, kBackwardWarps * 32, smem, 1, stream, a, run);
    });
}

} // namespace ep
