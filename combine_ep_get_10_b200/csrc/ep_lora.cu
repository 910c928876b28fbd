// ep_lora.cu -- low-rank adapters on the rows of a token-choice layout.
//
// The layout groups rows by adapter, so a tile of rows of one group is an
// ordinary matrix product with that adapter's factors: the rows are read where
// they are (row_token, or the dispatched rows themselves).  Three products, all
// bound by memory at the ranks they are for (4 rank flops a byte of row data
// and less; the tensor cores are busy 10 to 15 % of the time at rank 32):
//   shrink  u = s_e X W        long sum over the hidden width, rank columns
//   expand  out = base + u W   rank-long sum, hidden columns, base and out move
//   outer   dW = sum of rows   sum over a group's rows
// All on tcgen05 with bf16 operands and fp32 sums in tensor memory; u (fp32)
// enters as three bf16 terms (ep_mma.cuh), which keep all of its 24 bits.  The
// tensor core cuts a sum, where fp32 arithmetic rounds it: n additions in a row
// are off by about n / 4 * 2^-24, all towards zero (256: 4e-6).  So a chain has 16
// products, and chains are added up in fp32 registers.  Where adapters have
// few rows, a kernel of its own does shrink and expand at once (few).
//
// Rows come by cp.async, 16 bytes a lane: as fast for 128 bytes a row at a time
// as for 512 (4.75 TB/s for 4096 x 7168 read, 5.2 TB/s read and written), and
// any row may be anywhere.  Factors come through tensor maps, which lay them
// out as the tensor core reads them and fill what is past the rank, the width
// or the last column with zeros.
//
// Tensor memory is never waited for: no CTAs of these kernels that fit an SM
// together need more than its 512 columns.
//
// The kernels of a call are programmatic dependents of one another: what does
// not depend on the kernel before (which rows, the first tiles of base and of
// the factors) is done while that one runs.  Only the products' own results are
// read after the wait, through L2.
#include <algorithm>
#include <atomic>
#include <utility>

#include <cooperative_groups.h>

#include "ep_lora_launch.h"
#include "ep_mma.cuh"
#include "ep_tcgen05.cuh"
#include "ep_tma.cuh"

namespace ep {

namespace cg = cooperative_groups;

namespace {

constexpr int kRowTile = 64; // rows without an adapter that a CTA copies

// ------------------------------------------------------------------- rows
struct RowRange {
    int begin, end;
};

// Rows of adapter e, within [0, num_rows).
__device__ __forceinline__ RowRange group_rows(const LoraRows& g, int e)
{
    if (g.mode == EP_LAYOUT_COMPACT) {
        const int b = min(max(__ldg(g.offsets + e), 0), g.num_rows);
        return {b, max(min(__ldg(g.offsets + e + 1), g.num_rows), b)};
    }
    const int64_t b = min(static_cast<int64_t>(e) * g.max_tokens, static_cast<int64_t>(g.num_rows));
    const int64_t n = min(max(min(__ldg(g.counts + e), g.max_tokens), 0), g.num_rows - static_cast<int>(b));
    return {static_cast<int>(b), static_cast<int>(b + n)};
}

// The adapters that a lane has of a call's, `per` consecutive ones: the rows of
// the first kHeld (all of them up to 256 adapters) stay in registers.
struct LaneGroups {
    static constexpr int kHeld = 8;
    int e0, per; // adapters e0 .. e0 + per - 1
    RowRange held[kHeld];

    __device__ __forceinline__ LaneGroups(const LoraRows& g, int lane)
    {
        const int most = (g.E + 31) / 32;
        e0 = min(lane * most, g.E);
        per = min(most, g.E - e0);
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < per)
                held[j] = group_rows(g, e0 + j);
    }
    // f(adapter, its rows) for each of the lane's; f returns true to stop.
    template <typename F>
    __device__ __forceinline__ void each(const LoraRows& g, F&& f) const
    {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            if (j >= per)
                return;
            if (f(e0 + j, held[j]))
                return;
        }
        for (int j = kHeld; j < per; ++j)
            if (f(e0 + j, group_rows(g, e0 + j)))
                return;
    }
};

// Does the layout have more rows than the routing has pairs: the grids are for
// those, so none of its rows is worked on, by any kernel of the call.  mine: the
// lane's share of them.  One warp.
__device__ __forceinline__ bool too_many_rows(const LoraRows& g, int64_t mine)
{
    const int64_t most = g.pairs + 1; // at most 2^24 + 1: 32 lanes' fit
    return __reduce_add_sync(kFullMask, static_cast<uint32_t>(mine < most ? mine : most)) > static_cast<uint32_t>(g.pairs);
}

// The lane in whose run of `n` item i lies, and the items before that lane's;
// -1 when there are fewer items.  One warp.
__device__ __forceinline__ int find_lane(int n, int i, int lane, int& before)
{
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFullMask, inc, d);
        if (lane >= d)
            inc += o;
    }
    const uint32_t past = __ballot_sync(kFullMask, inc > i);
    before = inc - n;
    return past == 0u ? -1 : __ffs(past) - 1;
}

// Tiles of TILE rows are numbered adapter after adapter: the adapter and rows of
// tile i; false when there are fewer.  One warp; all lanes get the answer.
template <int TILE>
__device__ __forceinline__ bool find_tile(const LoraRows& g, int i, int lane, int& e, RowRange& rows)
{
    const LaneGroups groups(g, lane);
    const auto tiles = [](const RowRange& r) { return (r.end - r.begin + TILE - 1) / TILE; };
    int n = 0;
    int64_t all = 0;
    groups.each(g, [&](int, const RowRange& r) {
        n += tiles(r);
        all += r.end - r.begin;
        return false;
    });
    int before;
    const int from = find_lane(n, i, lane, before);
    if (from < 0 || too_many_rows(g, all))
        return false;
    int found = 0, left = i - before;
    RowRange mine{0, 0};
    if (lane == from)
        groups.each(g, [&](int j, const RowRange& r) {
            const int t = tiles(r);
            if (left >= t) {
                left -= t;
                return false;
            }
            found = j;
            mine.begin = r.begin + left * TILE;
            mine.end = min(r.end, mine.begin + TILE);
            return true;
        });
    e = __shfl_sync(kFullMask, found, from);
    rows.begin = __shfl_sync(kFullMask, mine.begin, from);
    rows.end = __shfl_sync(kFullMask, mine.end, from);
    return true;
}

// Rows that the routing fills past num_rows are left out, and all rows where the
// layout has more than the routing has pairs (it is another routing's, or the
// routing is a part of the layout's); the first CTA of a call's first
// kernel says so.  One warp.
__device__ __forceinline__ void report_overflow(const LoraRows& g, int lane)
{
    bool over = false;
    int64_t total = 0;
    for (int e = lane; e < g.E; e += 32) {
        if (g.mode == EP_LAYOUT_COMPACT) {
            const int end = __ldg(g.offsets + e + 1);
            over = over || end > g.num_rows;
            total += end - __ldg(g.offsets + e);
        } else {
            const int n = __ldg(g.counts + e);
            over = over || n > g.max_tokens || (n > 0 && static_cast<int64_t>(e) * g.max_tokens + n > g.num_rows);
            total += n;
        }
    }
    for (int d = 16; d >= 1; d >>= 1)
        total += __shfl_xor_sync(kFullMask, total, d);
    if (over || total > g.pairs)
        flag_error(g.err, EP_DEVERR_OVERFLOW);
}

// A call without row buffer: what there is to say about its rows.
__global__ void overflow_kernel(LoraRows g)
{
    pdl_wait();
    report_overflow(g, threadIdx.x & 31);
}

// Most tiles that the rows can make: a full one for every `tile` rows and a part
// one for every adapter in use.
int most_tiles(const LoraRows& g, int tile)
{
    const int rows = std::min(g.pairs, g.num_rows);
    return rows / tile + std::min(g.E, rows);
}

// Where the data of `row` is, in two steps so that the table's entry can be on
// its way while other work is done: the entry (-1 past the group's end), and the
// row index in x, base or out (-1 for an entry that is none).
__device__ __forceinline__ int row_entry(const LoraRows& g, int row, int end)
{
    int entry = row < end ? row : -1;
    // predicated, into entry itself: a load in a branch would be copied at the
    // branch's end, and the copy would wait for it
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
                 : "+r"(entry)
                 : "l"(g.row_token + row), "r"(g.row_token != nullptr && row < end ? 1u : 0u));
    return entry;
}

__device__ __forceinline__ int row_index(const LoraRows& g, int entry, int row, int end)
{
    if (row >= end || g.row_token == nullptr)
        return entry;
    if (entry < 0 || entry >= g.T) {
        flag_error(g.err, EP_DEVERR_BAD_INDEX);
        return -1;
    }
    return entry;
}

__device__ __forceinline__ int row_at(const LoraRows& g, int row, int end)
{
    return row_index(g, row_entry(g, row, end), row, end);
}

// ------------------------------------------------------------------ shrink
constexpr int kShrinkTile = 64; // rows
constexpr int kDepth = 128;     // hidden channels a stage, in tiles of 64
constexpr int kShrinkChain = 2; // stages whose products are summed in tensor memory

template <int RP>
struct ShrinkShape {
    // warps 0 .. 3 load x, 4 and 5 (and 8 and 9: the upper half of the ranks) add the
    // chains up, 6 multiplies, 7 loads w
    static constexpr int kSumWarps = RP <= 32 ? 2 : 4;
    static constexpr int kThreads = RP <= 32 ? 256 : 320;
    static constexpr int kCtas = RP <= 32 ? 4 : 3;             // 64 registers, so that two leave room for an expand CTA
    static constexpr int kSumRanks = RP / (kSumWarps / 2);     // a warp of those
    // in its registers, else in tensor memory (all ranks there: prefill 51.7 us, not 51.1)
    static constexpr bool kHeld = kSumRanks <= 32;
    static constexpr int kPlaces = kHeld ? 2 : 1;              // for chains, in tensor memory
    static constexpr int kStages = RP <= 32 ? 4 : (RP == 64 ? 3 : 2); // two CTAs an SM
    static constexpr int kHalfBytes = kShrinkTile * 128; // 64 channels of x
    static constexpr int kXBytes = kShrinkTile * kDepth * 2;
    static constexpr int kWBytes = RP * kDepth * 2;
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kPitch = RP + 4; // floats a row of the partial sums
    static constexpr int kSumBytes = kShrinkTile * kPitch * 4;
    // tiles start on 1024 bytes; a product reads 128 rows from a stage's first on
    static constexpr int kBehind = kHalfBytes - kWBytes; // past the last stage
    static constexpr int kBytes = kStages * kStageBytes + (kBehind > 0 ? kBehind : 0) + 1024;
    static_assert(kSumBytes <= kStages * kStageBytes, "the sums take the stages' place");
    static constexpr int kCols = 2 * RP; // tensor memory: two chains' sums, or one's and those before
    static constexpr Swizzle kSwizzle = RP == 16 ? Swizzle::k32 : (RP == 32 ? Swizzle::k64 : Swizzle::k128);
    static constexpr int kWBox = RP < 64 ? RP : 64; // ranks a box of w [K, rank]
};

// Bound by the rows' bytes: 4096 x 7168, 8 adapters of rank 32, 17 us with the
// launch (59 MB, 3.4 TB/s; a kernel that only copies such rows 12.4 us).  What is
// left are the ends: 2 us to find the tile and its rows, 2 us for the sums.
//
// A cluster has one tile of rows; its CTAs split the hidden width, and each
// adds up its share of the tile's rows over the cluster, in CTA order (the
// same sum every time, no atomics, no partial sums in HBM).  Four warps copy
// the rows of x from where they are, a thread brings the factor's slice, and
// another multiplies from shared memory into tensor memory: what is in flight is
// bounded by the stages alone.  Chains of kShrinkChain stages alternate between two
// places in tensor memory; while one is summed, two warps (rows 0 .. 31 and 32 .. 63)
// add the other one to their registers, or, where that takes too many of them, to a
// sum in tensor memory.  The product has 128 rows: what lies behind a stage's 64
// gives sums that nobody reads.
template <int RP, bool TRANS>
__global__ void __launch_bounds__(ShrinkShape<RP>::kThreads, ShrinkShape<RP>::kCtas)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap w_map, LoraShrinkLaunch a)
{
    using S = ShrinkShape<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[S::kStages], s_free[S::kStages], s_sums[2], s_taken[2];
    __shared__ uint32_t s_tmem;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_addr(smem);
    if (tid == 0) {
        prefetch_map(&w_map);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s_full[i], 129);
            mbar_init(&s_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_sums[i], 1);
            mbar_init(&s_taken[i], S::kSumWarps);
        }
        fence_mbar_init();
    }
    pdl_wait();
    if (a.trigger_dependents != 0)
        pdl_launch_dependents();
    if (blockIdx.x == 0 && warp == 0)
        report_overflow(a.rows, lane);
    int e;
    RowRange rows;
    if (!find_tile<kShrinkTile>(a.rows, blockIdx.x / parts, lane, e, rows))
        return; // the whole cluster has the same tile
    const int live = rows.end - rows.begin;
    const int steps = (a.K + kDepth - 1) / kDepth;
    const int n = (steps - part + parts - 1) / parts; // steps part, part + parts, ..: the cluster reads along the rows
    // 16-byte chunk tid % 16 of rows tid / 16 + 8 j (warps 0 .. 3); rows past the
    // group's end are left out (what their rows of the product hold is not
    // used), rows without data are zeros in every stage
    const int c = tid % 16;
    const uint32_t to = base + (c >> 3) * S::kHalfBytes + swizzled<8>((tid / 16) & 7, c & 7); // + 1024 j
    const uint16_t* x_row[8];
    uint32_t on = 0u; // rows with data
    if (warp < 4) {
        int entry[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            entry[j] = row_entry(a.rows, rows.begin + tid / 16 + 8 * j, rows.end);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = rows.begin + tid / 16 + 8 * j;
            const int at = row_index(a.rows, entry[j], row, rows.end);
            on |= (at >= 0 ? 1u : 0u) << j;
            x_row[j] = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(max(at, 0)) * a.K + c * 8 + part * kDepth;
            if (at < 0 && row < rows.end)
                for (int i = 0; i < S::kStages; ++i)
                    sts_v4(to + i * S::kStageBytes + 1024u * j, make_uint4(0u, 0u, 0u, 0u));
        }
        fence_proxy_async_shared();
    }
    if (warp == 6)
        tmem_alloc(&s_tmem, S::kCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem;

    const bool sums_up = warp == 4 || warp == 5 || warp >= 8;
    const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 1) * 32) << 16) + (warp >= 8 ? S::kSumRanks : 0);
    float total[S::kHeld ? S::kSumRanks : 1];
    bool alive = true; // no wait has run out
    if (warp < 4) {
        for (int i = 0; i < n; ++i) {
            const int stage = i % S::kStages;
            if (i >= S::kStages && alive)
                alive = mbar_wait_bounded(&s_free[stage], (i / S::kStages - 1) & 1, a.rows.err);
            const uint32_t bytes = (part + i * parts) * kDepth + c * 8 < a.K ? 16 : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if ((on >> j & 1u) != 0u)
                    cp_async16(to + stage * S::kStageBytes + 1024u * j, x_row[j], bytes);
                x_row[j] += parts * kDepth;
            }
            cp_async_arrive(&s_full[stage]);
        }
        cp_async_wait_all();
    } else if (warp == 7) {
        for (int i = 0; lane == 0 && i < n; ++i) {
            const int stage = i % S::kStages, k = (part + i * parts) * kDepth;
            if (i >= S::kStages && !mbar_wait_bounded(&s_free[stage], (i / S::kStages - 1) & 1, a.rows.err))
                break;
            const uint32_t ws = base + stage * S::kStageBytes + S::kXBytes;
            mbar_arrive_expect_tx(&s_full[stage], S::kWBytes);
            if (!TRANS) {
                tma_load3(ws, &w_map, k, 0, e, &s_full[stage]);
                tma_load3(ws + RP * 128, &w_map, k + 64, 0, e, &s_full[stage]);
            } else {
#pragma unroll
                for (int j = 0; j < RP; j += S::kWBox)
                    tma_load3(ws + j * kDepth * 2, &w_map, j, k, e, &s_full[stage]);
            }
        }
    } else if (sums_up) {
        if (S::kHeld) {
#pragma unroll
            for (int j = 0; j < S::kSumRanks; ++j)
                total[j] = 0.0f;
        }
        for (int chain = 0; chain * kShrinkChain < n; ++chain) {
            const int place = chain % S::kPlaces;
            if (alive)
                alive = mbar_wait_bounded(&s_sums[place], (chain / S::kPlaces) & 1, a.rows.err);
            tc_fence_after_sync();
            if constexpr (S::kHeld) {
#pragma unroll
                for (int j = 0; j < S::kSumRanks; j += 16) {
                    float d[16];
                    tmem_load16(d, mine + place * RP + j);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        total[j + i] += d[i];
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < S::kSumRanks; j += 16) {
                    float d[16];
                    tmem_load16(d, mine + j);
                    if (chain > 0) {
                        float before[16];
                        tmem_load16(before, mine + RP + j);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            d[i] += before[i];
                    }
                    tmem_store16(mine + RP + j, d);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s_taken[place]);
        }
    } else if (lane == 0) {
        constexpr uint32_t desc = product_desc(128, RP, false, TRANS);
        for (int i = 0; i < n; ++i) {
            const int stage = i % S::kStages, chain = i / kShrinkChain, link = i % kShrinkChain;
            if (!mbar_wait_bounded(&s_full[stage], (i / S::kStages) & 1, a.rows.err))
                break;
            const int place = chain % S::kPlaces;
            if (link == 0 && chain >= S::kPlaces &&
                !mbar_wait_bounded(&s_taken[place], (chain / S::kPlaces - 1) & 1, a.rows.err))
                break;
            fence_proxy_async_shared(); // the copies were the other threads'
            tc_fence_after_sync();
            const uint32_t xs = base + stage * S::kStageBytes, ws = xs + S::kXBytes;
#pragma unroll
            for (int kk = 0; kk < kDepth / 16; ++kk) {
                const uint64_t xd = operand_desc(xs + kk / 4 * S::kHalfBytes + kk % 4 * 32, Swizzle::k128, 0, 1024);
                const uint64_t wd = TRANS ? operand_desc(ws + kk * 2 * S::kWBox * 16, S::kSwizzle, kDepth * S::kWBox * 2,
                                                         S::kWBox * 16)
                                          : operand_desc(ws + kk / 4 * RP * 128 + kk % 4 * 32, Swizzle::k128, 0, 1024);
                tc_product(tmem + place * RP, xd, wd, desc, link > 0 || kk > 0);
            }
            if (i + S::kStages < n)
                tc_commit(&s_free[stage]);
            if (link == kShrinkChain - 1 || i == n - 1)
                tc_commit(&s_sums[place]);
        }
    }
    __syncwarp();
    __syncthreads(); // the last chain has been added: no product reads the stages any more

    // the tile's partial sums to shared memory, then the cluster's sums of them
    float* sums = reinterpret_cast<float*>(smem);
    if (sums_up) {
        float* row = sums + ((warp & 1) * 32 + lane) * S::kPitch + (warp >= 8 ? S::kSumRanks : 0);
        const auto store4 = [&](int j, const float* v) { *reinterpret_cast<float4*>(row + j) = make_float4(v[0], v[1], v[2], v[3]); };
        if constexpr (S::kHeld) {
#pragma unroll
            for (int j = 0; j < S::kSumRanks; j += 4)
                store4(j, total + j);
        } else {
#pragma unroll 1
            for (int j = 0; j < S::kSumRanks; j += 16) {
                float d[16];
                tmem_load16(d, mine + RP + j);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    store4(j + i, d + i);
            }
            tc_fence_before_sync();
        }
    }
    cluster.sync();
    if (warp == 6)
        tmem_free(tmem, S::kCols);
    const float scale = a.scales != nullptr ? __ldg(a.scales + e) : 1.0f;
    const int vecs = a.rank / 4;
    for (int i = part * S::kThreads + tid; i < live * vecs; i += parts * S::kThreads) {
        const int row = i / vecs, v = i - row * vecs;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = 0; c < parts; ++c) {
            const float4 o = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, c) + row * S::kPitch + 4 * v);
            s.x += o.x;
            s.y += o.y;
            s.z += o.z;
            s.w += o.w;
        }
        *reinterpret_cast<float4*>(a.u + static_cast<int64_t>(rows.begin + row) * a.rank + 4 * v) =
            make_float4(scale * s.x, scale * s.y, scale * s.z, scale * s.w);
    }
    cluster.sync(); // no CTA leaves while its sums are read
}

// ------------------------------------------------------------------ expand
constexpr int kExpandThreads = 288; // eight warps that add and store, one that loads w and multiplies
constexpr int kExpandTile = 128;    // rows: the product's M
constexpr int kExpandCols = 64;     // columns a step: the product's N
constexpr int kExpandGrid = 2 * 148; // two CTAs an SM, the first beside the shrink's

// A CTA's share of a call: one tile of rows, and every parts-th column step of
// it from step `part` on.
struct ExpandShare {
    RowRange rows;
    int e, part, parts;
};

// Share i; false when there are fewer.  A step is taken to cost as its live rows
// and kStepRows more; each tile gets shares for its part of the whole, rounded
// up, so that kExpandGrid CTAs are enough (with one share a tile where there are
// more tiles than that).  One warp; all lanes get the answer.
__device__ __forceinline__ bool find_share(const LoraRows& g, int i, int steps, int lane, ExpandShare& s)
{
    constexpr int kStepRows = 128; // 4096 rows of 16 adapters: 51 us, with 64 57 us, with 160 50 us
    const LaneGroups groups(g, lane);
    const auto tiles_of = [](const RowRange& r) { return (r.end - r.begin + kExpandTile - 1) / kExpandTile; };
    uint32_t cost = 0; // below 2^26: at most 2^24 rows
    uint32_t tiles = 0;
    int64_t all = 0;
    groups.each(g, [&](int, const RowRange& r) {
        all += r.end - r.begin;
        tiles += tiles_of(r);
        cost += r.end - r.begin + tiles_of(r) * kStepRows;
        return false;
    });
    if (too_many_rows(g, all))
        return false;
    tiles = __reduce_add_sync(kFullMask, tiles);
    cost = max(__reduce_add_sync(kFullMask, cost), 1u);
    const uint32_t spare = max(kExpandGrid - static_cast<int>(tiles), 0);
    const auto shares = [&](int rows) { // rounded down they add up to `spare` at most, and one a tile
        return min(steps, static_cast<int>((rows + kStepRows) * spare / cost) + 1);
    };
    const int full = shares(kExpandTile);
    const auto of = [&](const RowRange& r) { // of an adapter
        const int t = tiles_of(r);
        return t == 0 ? 0 : (t - 1) * full + shares(r.end - r.begin - (t - 1) * kExpandTile);
    };
    int n = 0;
    groups.each(g, [&](int, const RowRange& r) {
        n += of(r);
        return false;
    });
    int before;
    const int from = find_lane(n, i, lane, before);
    if (from < 0)
        return false;
    ExpandShare mine{};
    int left = i - before;
    if (lane == from)
        groups.each(g, [&](int j, const RowRange& r) {
            const int here = of(r);
            if (left >= here) {
                left -= here;
                return false;
            }
            const int tile = min(left / full, tiles_of(r) - 1);
            mine.e = j;
            mine.rows.begin = r.begin + tile * kExpandTile;
            mine.rows.end = min(r.end, mine.rows.begin + kExpandTile);
            mine.part = left - tile * full;
            mine.parts = shares(mine.rows.end - mine.rows.begin);
            return true;
        });
    s.e = __shfl_sync(kFullMask, mine.e, from);
    s.rows.begin = __shfl_sync(kFullMask, mine.rows.begin, from);
    s.rows.end = __shfl_sync(kFullMask, mine.rows.end, from);
    s.part = __shfl_sync(kFullMask, mine.part, from);
    s.parts = __shfl_sync(kFullMask, mine.parts, from);
    return true;
}

// out = base for those of kRowTile tokens from t0 on that have no adapter, by
// eight warps.
__device__ __forceinline__ void copy_base_rows(const LoraRows& g, const int32_t* slot, const void* base, void* out, int N,
                                               int t0, int warp, int lane)
{
    const int mine = t0 + (lane & 7) * 8 + warp;
    uint32_t todo = __ballot_sync(kFullMask, warp < 8 && lane < 8 && mine < g.T && __ldg(slot + mine) < 0);
    for (; todo != 0u; todo &= todo - 1u) {
        const int64_t at = static_cast<int64_t>(t0 + (__ffs(todo) - 1) * 8 + warp) * N;
#pragma unroll 4
        for (int c = lane * 8; c < N; c += 256) {
            const uint4 v = base != nullptr ? ld_nc_v4(static_cast<const uint16_t*>(base) + at + c)
                                            : make_uint4(0u, 0u, 0u, 0u);
            st_v4(static_cast<uint16_t*>(out) + at + c, v);
        }
    }
}

// The three terms of 8 consecutive values, `stride` bytes from term to term.
__device__ __forceinline__ void store_terms(uint8_t* to, int stride, float4 f0, float4 f1)
{
    uint32_t x[3], y[3], z[3], w[3];
    split_bf16x2(f0.x, f0.y, x);
    split_bf16x2(f0.z, f0.w, y);
    split_bf16x2(f1.x, f1.y, z);
    split_bf16x2(f1.z, f1.w, w);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint4*>(to + i * stride) = make_uint4(x[i], y[i], z[i], w[i]);
}

template <int RP>
struct ExpandShape {
    static constexpr int kTermBytes = kExpandTile * RP * 2; // one bf16 tile of u
    static constexpr int kWBytes = kExpandCols * RP * 2;
    static constexpr int kWStages = RP == 16 ? 6 : (RP == 32 ? 4 : 3); // three at least: one ahead of the step that loads
    static constexpr int kTileBytes = 8 * 32 * 64;          // base: 32 rows of 64 bytes a warp
    static constexpr int kTilesAt = 3 * kTermBytes + kWStages * kWBytes;
    static constexpr int kBytes = kTilesAt + 2 * kTileBytes + 1024; // operands start on 1024 bytes
    static constexpr Swizzle kSwizzle = RP == 16 ? Swizzle::k32 : (RP == 32 ? Swizzle::k64 : Swizzle::k128);
    static constexpr int kBox = RP < 64 ? RP : 64; // ranks a row of u's tiles, and of a box of w [N, rank]
};

__device__ __forceinline__ uint32_t add_to_bf16x2(uint32_t base, float a, float b)
{
    return pack_bf16x2(bf16_lo(base) + a, bf16_hi(base) + b);
}

// Bound by base and out: 4096 x 7168, 8 adapters of rank 32, 30 us after the
// product before it (117 MB, 4 TB/s; a copy of such rows alone 22.6 us).  A CTA
// that starts when the kernel before it ends needs 8 us to its first store, so
// the first of an SM's two starts beside the shrink's CTAs.
//
// A CTA has one tile of rows and every parts-th column step.  u stays in shared
// memory as three bf16 tiles, one a term; the small terms' products are summed
// first, so that few additions cut the large sum.  While one thread has the factor's next
// columns multiplied into one of two places in tensor memory, eight warps take the other one (32 rows and 32 columns each):
// a thread adds a row's sums to base in shared memory, then the warp stores its
// rows from there, four lanes 32 columns, and asks for base's tile after next.
template <int RP, bool TRANS>
__global__ void __launch_bounds__(kExpandThreads, RP <= 64 ? 2 : 1)
    lora_expand_kernel(const __grid_constant__ CUtensorMap w_map, LoraExpandLaunch a, int shares)
{
    using S = ExpandShape<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_w[S::kWStages], s_sums[2], s_taken[2];
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.after_u == 0)
        pdl_wait();
    if (static_cast<int>(blockIdx.x) >= shares) { // tokens without an adapter: out = base
        copy_base_rows(a.rows, a.slot, a.base, a.out, a.N, (blockIdx.x - shares) * kRowTile, warp, lane);
        pdl_wait();
        return;
    }
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t us = smem_addr(smem), ws0 = us + 3 * S::kTermBytes;
    if (tid == 256) {
        prefetch_map(&w_map);
        for (int i = 0; i < S::kWStages; ++i)
            mbar_init(&s_w[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_sums[i], 1);
            mbar_init(&s_taken[i], 8);
        }
        fence_mbar_init();
    }
    const int steps = (a.N + kExpandCols - 1) / kExpandCols;
    ExpandShare share;
    if (!find_share(a.rows, blockIdx.x, steps, lane, share)) {
        pdl_wait();
        return;
    }
    const RowRange rows = share.rows;
    const int e = share.e, part = share.part, parts = share.parts;
    const int n = (steps - part + parts - 1) / parts; // steps part, part + parts, ..

    const auto load_w = [&](int i) {
        uint64_t* bar = &s_w[i % S::kWStages];
        const uint32_t ws = ws0 + i % S::kWStages * S::kWBytes;
        const int n0 = (part + i * parts) * kExpandCols;
        mbar_arrive_expect_tx(bar, S::kWBytes);
        if (!TRANS) {
#pragma unroll
            for (int j = 0; j < RP; j += S::kBox)
                tma_load3(ws + j * kExpandCols * 2, &w_map, j, n0, e, bar);
        } else {
            tma_load3(ws, &w_map, n0, 0, e, bar);
        }
    };
    if (tid == 256)
        for (int i = 0; i < min(n, S::kWStages); ++i)
            load_w(i);

    // warp: rows 32 (warp % 4).., columns 32 (warp / 4)..; lane: rows lane / 4 + 8 r
    // of them, 8 columns from 8 (lane % 4) on
    const int q = warp & 3, ch = (warp >> 2) * 32;
    const bool busy = warp < 8 && rows.begin + 32 * q < rows.end;
    int at[4];
    const uint32_t mine = us + S::kTilesAt + warp * 2048;
    const uint32_t quad = mine + swizzled<4>(lane / 4, lane & 3); // + 512 r
    const auto load_base = [&](int i) {
        const int col = (part + i * parts) * kExpandCols + ch + (lane & 3) * 8;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool on = a.base != nullptr && at[r] >= 0 && col < a.N;
            const uint16_t* from = static_cast<const uint16_t*>(a.base) + static_cast<int64_t>(at[r]) * a.N + col;
            if (at[r] >= 0)
                cp_async16(quad + (i & 1) * S::kTileBytes + r * 512, on ? from : a.w, on ? 16 : 0);
        }
    };
    if (busy) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            at[r] = row_at(a.rows, rows.begin + 32 * q + lane / 4 + 8 * r, rows.end);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i < n)
                load_base(i);
            cp_async_commit();
        }
    }
    if (a.after_u == 1)
        pdl_wait();

    // u in three terms; rows past the group's end give sums that nobody reads
    const int live = rows.end - rows.begin;
    if (warp < 8) {
        const float* u = a.u + static_cast<int64_t>(rows.begin) * a.rank;
#pragma unroll 4
        for (int t = tid; t < live * (RP / 8); t += 256) {
            const int row = t / (RP / 8), c = t % (RP / 8);
            float4 f0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), f1 = f0;
            if (c * 8 < a.rank) {
                const float4* f = reinterpret_cast<const float4*>(u + static_cast<int64_t>(row) * a.rank + c * 8);
                f0 = __ldcg(f);
                f1 = __ldcg(f + 1);
            }
            const uint32_t place = (c >> 3) * (kExpandTile * 128u) + swizzled<S::kBox / 8>(row, c & 7);
            store_terms(smem + place, S::kTermBytes, f0, f1);
        }
        fence_proxy_async_shared();
    } else {
        tmem_alloc(&s_tmem, 2 * kExpandCols);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem;

    bool alive = true; // no wait has run out
    if (tid == 256) {
        constexpr uint32_t desc = product_desc(128, kExpandCols, false, TRANS);
        constexpr uint32_t group = S::kBox * 16; // 8 rows of u's tiles
        for (int i = 0; i < n && alive; ++i) {
            const int stage = i % S::kWStages;
            alive = mbar_wait_bounded(&s_w[stage], (i / S::kWStages) & 1, a.rows.err);
            if (i >= 2 && alive)
                alive = mbar_wait_bounded(&s_taken[i & 1], (i / 2 - 1) & 1, a.rows.err);
            if (!alive)
                break;
            tc_fence_after_sync();
            const uint32_t ws = ws0 + stage * S::kWBytes;
#pragma unroll
            for (int term = 2; term >= 0; --term)
#pragma unroll
                for (int kk = 0; kk < RP / 16; ++kk) {
                    const uint64_t x = operand_desc(us + term * S::kTermBytes + kk / 4 * kExpandTile * 128 + kk % 4 * 32,
                                                    S::kSwizzle, 0, group);
                    const uint64_t w = TRANS ? operand_desc(ws + kk * 2048, Swizzle::k128, 0, 1024)
                                             : operand_desc(ws + kk / 4 * kExpandCols * 128 + kk % 4 * 32, S::kSwizzle, 0, group);
                    tc_product(tmem + (i & 1) * kExpandCols, x, w, desc, term < 2 || kk > 0);
                }
            tc_commit(&s_sums[i & 1]); // frees w's stage too
            if (i >= 1 && i - 1 + S::kWStages < n) { // the step before is done, or nearly
                alive = mbar_wait_bounded(&s_sums[(i - 1) & 1], ((i - 1) / 2) & 1, a.rows.err);
                if (alive)
                    load_w(i - 1 + S::kWStages);
            }
        }
    } else if (warp < 8) {
        uint16_t* out = static_cast<uint16_t*>(a.out);
        for (int i = 0; i < n; ++i) {
            if (alive)
                alive = mbar_wait_bounded(&s_sums[i & 1], (i / 2) & 1, a.rows.err);
            tc_fence_after_sync();
            if (busy) {
                const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + (i & 1) * kExpandCols + ch;
                const uint32_t tile = (i & 1) * S::kTileBytes;
                cp_async_wait<1>();
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float d[16];
                    tmem_load16(d, from + 16 * h);
                    const uint32_t p0 = mine + tile + swizzled<4>(lane, 2 * h), p1 = mine + tile + swizzled<4>(lane, 2 * h + 1);
                    uint4 v0 = lds_v4(p0), v1 = lds_v4(p1);
                    v0 = make_uint4(add_to_bf16x2(v0.x, d[0], d[1]), add_to_bf16x2(v0.y, d[2], d[3]),
                                    add_to_bf16x2(v0.z, d[4], d[5]), add_to_bf16x2(v0.w, d[6], d[7]));
                    v1 = make_uint4(add_to_bf16x2(v1.x, d[8], d[9]), add_to_bf16x2(v1.y, d[10], d[11]),
                                    add_to_bf16x2(v1.z, d[12], d[13]), add_to_bf16x2(v1.w, d[14], d[15]));
                    sts_v4(p0, v0);
                    sts_v4(p1, v1);
                }
                tc_fence_before_sync();
                __syncwarp();
                const int col = (part + i * parts) * kExpandCols + ch + (lane & 3) * 8;
                uint4 v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[r] = lds_v4(quad + tile + r * 512);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (at[r] >= 0 && col < a.N)
                        st_v4(out + static_cast<int64_t>(at[r]) * a.N + col, v[r]);
                __syncwarp();
                if (i + 2 < n)
                    load_base(i + 2);
                cp_async_commit();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&s_taken[i & 1]);
        }
    }
    __syncthreads();
    if (warp == 8)
        tmem_free(tmem, 2 * kExpandCols);
    if (a.after_u == 2)
        pdl_wait(); // this grid ends after the one before it
}

// --------------------------------------------------------------------- few
constexpr int kFewThreads = 256;
constexpr int kFewTile = 16; // rows: the warp product's M
constexpr int kFewCluster = 8;
constexpr int kFewRank = 64; // largest rank

template <int RP>
struct FewShape {
    static constexpr int kRanks = 16;               // ranks a warp multiplies x with
    static constexpr int kRankWarps = RP / kRanks;  // warps side by side in them
    static constexpr int kWarpPitch = kRanks + 4;   // floats a row of a warp's sums
    static constexpr int kPitch = RP + 4;           // of the CTA's and the cluster's
    static constexpr int kWarpSums = kFewTile * kWarpPitch, kSums = kFewTile * kPitch; // floats
    static constexpr int kBytes = (8 * kWarpSums + 2 * kSums) * 4;
    static constexpr int kAhead = 4;                // blocks of 32 channels a warp loads at once
    static constexpr bool kTwo = RP <= 32;          // two groups of output columns on their way
};

// Both products of a forward call for a tile of 16 rows, where an adapter has few
// rows (a decode step): the bytes are the factors', each of them used once or
// read again from L2, and what lasts is latency.  A cluster has a tile; its warps split the hidden
// width, add their sums up over the cluster, and split the output columns.  One
// launch, no shared memory between HBM and the warp product, the first columns'
// factors and base on their way while u is added up: 128 rows of 64 adapters, all
// of them in use, rank 16, 7168 -> 4096, 10 us, with the two kernels for many rows
// 31 us.
//
// A sum may take its terms in any order, so a lane loads 16 consecutive bytes of
// a row of x and of the factor and calls them the product's columns k that it
// needs.  In the same way the columns of out are dealt to the products so that a
// thread ends with 8 consecutive ones.
template <int RP>
__global__ void __launch_bounds__(kFewThreads, 2) lora_few_kernel(LoraFewLaunch a, int tiles)
{
    using S = FewShape<RP>;
    extern __shared__ __align__(16) float s_few[];
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int unit = part * 8 + warp, units = parts * 8;
    pdl_wait();
    if (blockIdx.x == 0 && warp == 0)
        report_overflow(a.rows, lane);
    const int tile = blockIdx.x / parts;
    if (tile >= tiles) { // tokens without an adapter: out = base
        copy_base_rows(a.rows, a.slot, a.base, a.out, a.N, (blockIdx.x - tiles * parts) * kRowTile, warp, lane);
        return; // the whole cluster
    }
    int e;
    RowRange rows;
    if (!find_tile<kFewTile>(a.rows, tile, lane, e, rows))
        return;
    const int r0 = rows.begin + g, r1 = r0 + 8;
    const int entry0 = row_entry(a.rows, r0, rows.end), entry1 = row_entry(a.rows, r1, rows.end);
    const float scale = a.scales != nullptr ? __ldg(a.scales + e) : 1.0f;
    const uint16_t* wa = static_cast<const uint16_t*>(a.a) + static_cast<int64_t>(e) * a.rank * a.K;
    const uint16_t* wb = static_cast<const uint16_t*>(a.b) + static_cast<int64_t>(e) * a.rank * a.N;
    const int at0 = row_index(a.rows, entry0, r0, rows.end), at1 = row_index(a.rows, entry1, r1, rows.end);
    const uint16_t* x0 = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(max(at0, 0)) * a.K;
    const uint16_t* x1 = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(max(at1, 0)) * a.K;

    // u: ranks 16 (warp % kRankWarps).., every k_units-th block of 32 channels; lane:
    // 8 channels from 8 q
    const int j0 = warp % S::kRankWarps * S::kRanks;
    const int k_unit = part * (8 / S::kRankWarps) + warp / S::kRankWarps, k_units = parts * (8 / S::kRankWarps);
    float acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[j][i] = 0.0f;
    for (int k0 = k_unit * 32; k0 < a.K; k0 += S::kAhead * k_units * 32) {
        uint4 xa[S::kAhead][2], w[S::kAhead][2];
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i) {
            const int k = k0 + i * k_units * 32 + q * 8;
            const bool in = k < a.K;
            xa[i][0] = ld_nc_v4_if(x0 + k, in && at0 >= 0);
            xa[i][1] = ld_nc_v4_if(x1 + k, in && at1 >= 0);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[i][j] = ld_nc_v4_if(wa + static_cast<int64_t>(j0 + j * 8 + g) * a.K + k, in && j0 + j * 8 < a.rank);
        }
        float sum[2][4] = {}; // a chain of 8 products
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mma16816(sum[j], xa[i][0].x, xa[i][1].x, xa[i][0].y, xa[i][1].y, w[i][j].x, w[i][j].y);
                mma16816(sum[j], xa[i][0].z, xa[i][1].z, xa[i][0].w, xa[i][1].w, w[i][j].z, w[i][j].w);
            }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[j][i] += sum[j][i];
    }
    // base and the factor's rows of 32 columns: column 8 (n / 2) + 2 j + n % 2 is
    // row n of product j; a lane has 8 of each 32 ranks, of what is left 4 of 16
    // and 2 of 8
    struct Columns {
        uint4 base[2];
        uint2 w[RP / 16][4]; // of 16 ranks
    };
    const auto load_columns = [&](Columns& c, int group) {
        const int col = group * 32 + q * 8;
        const bool in = col < a.N && a.base != nullptr;
        const uint16_t* b = static_cast<const uint16_t*>(a.base) + col;
        c.base[0] = ld_v4_if(b + static_cast<int64_t>(max(at0, 0)) * a.N, in && at0 >= 0);
        c.base[1] = ld_v4_if(b + static_cast<int64_t>(max(at1, 0)) * a.N, in && at1 >= 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = group * 32 + 8 * (g / 2) + 2 * j + g % 2;
            const uint16_t* row = wb + static_cast<int64_t>(n) * a.rank;
#pragma unroll
            for (int s = 0; s < RP / 16; s += 2) {
                if (RP >= 32) {
                    const uint4 v = ld_nc_v4_if(row + s * 16 + q * 8, n < a.N && s * 16 + 32 <= a.rank);
                    c.w[s][j] = make_uint2(v.x, v.y);
                    c.w[(s + 1) % (RP / 16)][j] = make_uint2(v.z, v.w);
                }
                if (RP < 32 || s * 16 + 32 > a.rank) { // (uniform) not a whole block
                    const int whole = s * 16 + 16 <= a.rank ? 1 : 0; // steps of 16 in it
                    c.w[s][j] = ld_nc_v2_if(row + s * 16 + q * 4, n < a.N && whole == 1);
                    if (RP >= 32)
                        c.w[(s + 1) % (RP / 16)][j] = make_uint2(0u, 0u);
                    if (s * 16 + whole * 16 + 8 == a.rank) {
                        const uint32_t v = ld_nc_u32_if(row + (s + whole) * 16 + q * 2, n < a.N);
                        if (whole == 0)
                            c.w[s][j].x = v;
                        else if (RP >= 32)
                            c.w[(s + 1) % (RP / 16)][j].x = v;
                    }
                }
            }
        }
    };
    const int groups = (a.N + 31) / 32;
    Columns even, odd;
    load_columns(even, unit);
    if (S::kTwo)
        load_columns(odd, unit + units); // (past the last: zeros, and nothing is read)

    // the warps' sums, the CTA's, the cluster's: each in a fixed order
    float* s_cta = s_few + 8 * S::kWarpSums;
    float* s_u = s_cta + S::kSums;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float* p = s_few + warp * S::kWarpSums + g * S::kWarpPitch + j * 8 + 2 * q;
        *reinterpret_cast<float2*>(p) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(p + 8 * S::kWarpPitch) = make_float2(acc[j][2], acc[j][3]);
    }
    __syncthreads();
    const auto add4 = [](float4& to, const float4& v) {
        to.x += v.x;
        to.y += v.y;
        to.z += v.z;
        to.w += v.w;
    };
    for (int i = tid; i < kFewTile * RP / 4; i += kFewThreads) {
        const int row = i / (RP / 4), j = i % (RP / 4) * 4;
        const float* p = s_few + j / S::kRanks * S::kWarpSums + row * S::kWarpPitch + j % S::kRanks;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 8; w += S::kRankWarps)
            add4(sum, *reinterpret_cast<const float4*>(p + w * S::kWarpSums));
        *reinterpret_cast<float4*>(s_cta + row * S::kPitch + j) = sum;
    }
    cluster.sync();
    for (int i = tid; i < kFewTile * RP / 4; i += kFewThreads) {
        const int row = i / (RP / 4), j = i % (RP / 4) * 4, at = row * S::kPitch + j;
        float4 v[kFewCluster]; // all on their way at once
#pragma unroll
        for (int c = 0; c < kFewCluster; ++c)
            v[c] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(s_cta, min(c, parts - 1)) + at);
        float4 sum = v[0];
#pragma unroll
        for (int c = 1; c < kFewCluster; ++c)
            if (c < parts)
                add4(sum, v[c]);
        // ranks past the last are zeros (their rows of the factor count as zeros, but an
        // infinite x times those is no number)
        sum = j < a.rank ? make_float4(scale * sum.x, scale * sum.y, scale * sum.z, scale * sum.w)
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        *reinterpret_cast<float4*>(s_u + at) = sum;
        if (row % parts == part && j < a.rank && rows.begin + row < rows.end)
            *reinterpret_cast<float4*>(a.u + static_cast<int64_t>(rows.begin + row) * a.rank + j) = sum;
    }
    auto left = cluster.barrier_arrive(); // this CTA has read the others' sums
    __syncthreads();

    // out
    uint32_t u[RP / 16][4][3]; // in three terms
#pragma unroll
    for (int s = 0; s < RP / 16; ++s) {
        const bool half = s * 16 + 8 == a.rank, block = RP >= 32 && (s & ~1) * 16 + 32 <= a.rank;
        const int k = block ? (s & ~1) * 16 + q * 8 + (s & 1) * 4 : s * 16 + q * (half ? 2 : 4); // the lane's first rank
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float* p = s_u + (g + 8 * r) * S::kPitch + k;
            split_bf16x2(p[0], p[1], u[s][r]);
            split_bf16x2(half ? 0.0f : p[2], half ? 0.0f : p[3], u[s][2 + r]);
        }
    }
    uint16_t* out = static_cast<uint16_t*>(a.out);
    const auto finish = [&](Columns& c, int group) {
        float d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[j][i] = 0.0f;
#pragma unroll
            for (int term = 2; term >= 0; --term) // the small ones first
#pragma unroll
                for (int s = 0; s < RP / 16; ++s)
                    mma16816(d[j], u[s][0][term], u[s][1][term], u[s][2][term], u[s][3][term], c.w[s][j].x, c.w[s][j].y);
        }
        const uint4 b0 = c.base[0], b1 = c.base[1];
        load_columns(c, group + (S::kTwo ? 2 : 1) * units);
        const int col = group * 32 + q * 8;
        if (col >= a.N)
            return;
        if (at0 >= 0)
            st_v4(out + static_cast<int64_t>(at0) * a.N + col,
                  make_uint4(add_to_bf16x2(b0.x, d[0][0], d[0][1]), add_to_bf16x2(b0.y, d[1][0], d[1][1]),
                             add_to_bf16x2(b0.z, d[2][0], d[2][1]), add_to_bf16x2(b0.w, d[3][0], d[3][1])));
        if (at1 >= 0)
            st_v4(out + static_cast<int64_t>(at1) * a.N + col,
                  make_uint4(add_to_bf16x2(b1.x, d[0][2], d[0][3]), add_to_bf16x2(b1.y, d[1][2], d[1][3]),
                             add_to_bf16x2(b1.z, d[2][2], d[2][3]), add_to_bf16x2(b1.w, d[3][2], d[3][3])));
    };
    for (int group = unit; group < groups; group += (S::kTwo ? 2 : 1) * units) {
        finish(even, group);
        if (S::kTwo && group + units < groups)
            finish(odd, group + units);
    }
    cluster.barrier_wait(std::move(left)); // no CTA leaves while its sums are read
}

// ------------------------------------------------------------------- outer
constexpr int kOuterThreads = 320; // four warps that load x or dy, four that split u and store, one that multiplies, one that loads u
constexpr int kOuterRows = 64;     // rows a stage
constexpr int kOuterCols = 128;    // columns of x or dy a tile: the product's M
constexpr int kOuterParts = 4;     // CTAs that share a tile's rows, at most
constexpr int kOuterChain = 4;     // stages whose products are summed in tensor memory

template <int RP>
struct OuterShape {
    static constexpr int kHalfBytes = kOuterRows * 128;    // 64 columns of x or dy, or of u's terms
    static constexpr int kVBytes = kOuterRows * kOuterCols * 2;
    static constexpr int kTermBytes = kOuterRows * RP * 2;
    static constexpr int kUBytes = 3 * kTermBytes;         // u as it is in HBM, then its three terms
    // Three CTAs an SM as far as the rank allows, the stages of a CTA in 72 KB: all
    // gradients of 4096 rows, rank 32, 80 us, with two CTAs and 87 KB 96 us.
    static constexpr int kCtas = RP <= 32 ? 3 : (RP == 64 ? 2 : 1);
    static constexpr int kStages = RP == 128 ? 4 : 3;  // of x or dy
    static constexpr int kUStages = RP == 16 || RP == 128 ? 3 : 2; // of u
    static constexpr int kUAt = kStages * kVBytes;
    static constexpr int kBytes = kUAt + kUStages * kUBytes + 1024; // tiles start on 1024 bytes
    static constexpr int kPitch = RP + 4;                       // floats a column of a part's sums
    static_assert(kOuterCols * kPitch * 4 + 1024 <= kBytes, "a part's sums take the stages' place");
    static constexpr int kTmem = 4 * RP;                        // the three terms' sums, the chains' before
    static constexpr int kSide = RP <= 64 ? 3 : 2; // terms that one product takes side by side (256 columns at most)
    static constexpr Swizzle kSwizzle = RP == 16 ? Swizzle::k32 : (RP == 32 ? Swizzle::k64 : Swizzle::k128);
    static constexpr int kUChunks = RP < 64 ? RP / 8 : 8; // 16-byte chunks a row of u's terms
};

// Place of columns 8c.. of `row` in a tile of 128-byte rows, 64 columns each.
__device__ __forceinline__ uint32_t in_halves(int row, int c)
{
    return static_cast<uint32_t>(c >> 3) * (kOuterRows * 128u) + swizzled<8>(row, c & 7);
}

// The output tiles of a call: adapter after adapter, in each the column tiles of
// db and then of da.  Up to 32 adapters are taken in the order of their rows,
// most first; CTAs take tiles in turn, forth and back, so that each gets long
// and short ones.  Where there are fewer tiles than places, a cluster has a tile,
// its CTAs a part of the tile's stages each.
struct OuterTile {
    RowRange rows;
    int e, n0, stages;
    bool in; // da, from x and dh; else db, from dy and h
};

template <bool SPLIT>
struct OuterTiles {
    int in_tiles, out_tiles, total;
    int parts, part, places, place; // CTAs a tile, which of them; clusters, which of them
    int adapter;   // lane i: the i-th adapter by rows
    RowRange rows; // and its rows
    bool none;     // no rows at all (too_many_rows)

    // One warp.
    __device__ __forceinline__ OuterTiles(const LoraRows& g, int in_tiles_, int out_tiles_, int parts_, int lane)
        : in_tiles(in_tiles_), out_tiles(out_tiles_), total(g.E * (in_tiles_ + out_tiles_)), parts(SPLIT ? parts_ : 1),
          part(SPLIT ? static_cast<int>(blockIdx.x) % parts_ : 0),
          places(static_cast<int>(gridDim.x) / (SPLIT ? parts_ : 1)),
          place(static_cast<int>(blockIdx.x) / (SPLIT ? parts_ : 1)), adapter(0), rows{0, 0}
    {
        int64_t all = 0;
        if (g.E > 32) {
            for (int e = lane; e < g.E; e += 32) {
                const RowRange r = group_rows(g, e);
                all += r.end - r.begin;
            }
            none = too_many_rows(g, all);
            return;
        }
        RowRange mine{0, -1};
        if (lane < g.E)
            mine = group_rows(g, lane);
        none = too_many_rows(g, max(mine.end - mine.begin, 0));
        const int n = mine.end - mine.begin;
        int before = 0;
        for (int j = 0; j < g.E; ++j) {
            const int o = __shfl_sync(kFullMask, n, j);
            before += o > n || (o == n && j < lane) ? 1 : 0;
        }
        for (int j = 0; j < g.E; ++j) {
            const int place = __shfl_sync(kFullMask, before, j);
            adapter = place == lane ? j : adapter;
        }
        rows.begin = __shfl_sync(kFullMask, mine.begin, adapter);
        rows.end = __shfl_sync(kFullMask, mine.end, adapter);
    }
    // Tile k of this CTA; false for none (a later one may be).  One warp.
    __device__ __forceinline__ bool get(const LoraRows& g, int k, OuterTile& t) const
    {
        const int i = k * places + ((k & 1) != 0 ? places - 1 - place : place);
        if (i >= total)
            return false;
        const int per = in_tiles + out_tiles, at = i / per, tile = i - at * per;
        t.in = tile >= out_tiles;
        t.n0 = (t.in ? tile - out_tiles : tile) * kOuterCols;
        if (g.E > 32) {
            t.e = at;
            t.rows = group_rows(g, at);
        } else {
            t.e = __shfl_sync(kFullMask, adapter, at);
            t.rows.begin = __shfl_sync(kFullMask, rows.begin, at);
            t.rows.end = __shfl_sync(kFullMask, rows.end, at);
        }
        if (none)
            t.rows.end = t.rows.begin;
        t.stages = (t.rows.end - t.rows.begin + kOuterRows - 1) / kOuterRows;
        if (SPLIT) {
            const int mine = (t.stages + parts - 1) / parts;
            t.rows.begin = min(t.rows.begin + part * mine * kOuterRows, t.rows.end);
            t.rows.end = min(t.rows.end, t.rows.begin + mine * kOuterRows);
            t.stages = (t.rows.end - t.rows.begin + kOuterRows - 1) / kOuterRows;
        }
        return true;
    }
    __device__ __forceinline__ int rounds() const { return (total + places - 1) / places; }
};

// The four warps that split u.
__device__ __forceinline__ void split_warps_sync()
{
    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}

__device__ __forceinline__ bool split_warps_any(bool mine)
{
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(mine ? 1u : 0u)
                 : "memory");
    return any != 0u;
}

// Bound by x and dy: 4096 x 7168 each, 8 adapters of rank 32, 34 us after the
// product before it (117 MB, 3.5 TB/s), and by the chains that turn u into its
// terms, of which three CTAs an SM hide most (rank 64, two CTAs: 61 us; rank 128,
// one: 139 us).
//
// dW of one adapter and kOuterCols columns of x or dy, tile after tile: the
// columns are the product's rows (M), the rank its columns (N), and the sum
// runs over the adapter's rows, kOuterRows a stage.  Both operands are MN-major:
// the row data as it lies in HBM, and u, copied as fp32 and turned in place into
// three bf16 tiles that one product takes side by side (at the largest rank two
// do).  Sums stay in tensor memory: the terms' and, apart, those of the chains
// before, to which the warps that split u add a chain when it is done.  The warps
// that load run on into the next tile's stages while a tile is stored.
template <int RP, bool SPLIT>
__global__ void __launch_bounds__(kOuterThreads, RP <= 64 ? 3 : 1) // (64 registers for three)
    lora_outer_kernel(LoraOuterLaunch a, int in_tiles, int out_tiles, int parts)
{
    using S = OuterShape<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_v[S::kStages], s_free[S::kStages], s_u[S::kUStages], s_split[S::kUStages], s_done, s_taken;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_addr(smem);
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s_v[i], 128);
            mbar_init(&s_free[i], 1);
        }
        for (int i = 0; i < S::kUStages; ++i) {
            mbar_init(&s_u[i], 1);
            mbar_init(&s_split[i], 128);
        }
        mbar_init(&s_done, 1);
        mbar_init(&s_taken, 4);
        fence_mbar_init();
    }
    pdl_wait();
    if (a.trigger_dependents != 0)
        pdl_launch_dependents(); // what comes next needs dh, which is there
    if (warp == 8)
        tmem_alloc(&s_tmem, S::kTmem);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    const OuterTiles<SPLIT> tiles(a.rows, in_tiles, out_tiles, parts, lane);
    const int rounds = tiles.rounds();
    OuterTile t;
    bool alive = true; // no wait has run out
    int at_stage = 0;  // stages so far, over all tiles
    int chains = 0;    // chains waited for so far, over all tiles
    const auto stage_free = [&](int stages) { // the products that read the place in a ring of `stages` before are done
        const int before = at_stage - stages;
        if (before >= 0 && alive)
            alive = mbar_wait_bounded(&s_free[before % S::kStages], (before / S::kStages) & 1, a.rows.err);
    };

    if (warp < 4) {
        // 16-byte chunk tid % 16 of rows tid / 16 + 8 j; lanes 0 .. 15 look up the
        // rows of the warp's two half rows: j = lane / 2 of half warp lane % 2
        const int c = tid % 16, r0 = tid / 16;
        const uint32_t to = in_halves(r0, c); // + 1024 j
        const int mine = warp * 2 + (lane & 1) + 8 * (lane / 2);
        for (int k = 0; k < rounds; ++k) {
            if (!tiles.get(a.rows, k, t))
                continue;
            const int N = t.in ? a.hidden_in : a.hidden_out;
            const uint16_t* v = static_cast<const uint16_t*>(t.in ? a.x : a.dy);
            const bool in_col = t.n0 + c * 8 < N;
            const uint16_t* from = in_col ? v + t.n0 + c * 8 : v;
            const int end = lane < 16 ? t.rows.end : 0;
            const auto find = [&](int i) { return row_entry(a.rows, t.rows.begin + i * kOuterRows + mine, end); };
            const auto load = [&](int i, int& entry) {
                const int index = row_index(a.rows, entry, t.rows.begin + i * kOuterRows + mine, end);
                entry = find(i + 2);
                stage_free(S::kStages);
                int at[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    at[j] = __shfl_sync(kFullMask, index, j * 2 + (r0 & 1));
                const uint32_t vs = base + at_stage % S::kStages * S::kVBytes + to;
#pragma unroll
                for (int j = 0; j < 8; ++j) // rows that are none, and columns past the last, are zeros
                    cp_async16(vs + 1024u * j, from + static_cast<int64_t>(max(at[j], 0)) * N,
                               at[j] >= 0 && in_col ? 16 : 0);
                cp_async_arrive(&s_v[at_stage % S::kStages]);
                ++at_stage;
            };
            int even = find(0), odd = find(1); // entries of the stage at hand and of the next one
            for (int i = 0; i < t.stages; i += 2) {
                load(i, even);
                if (i + 1 < t.stages)
                    load(i + 1, odd);
            }
        }
        cp_async_wait_all();
    } else if (warp == 9) {
        for (int k = 0; k < rounds; ++k) {
            if (!tiles.get(a.rows, k, t) || lane != 0)
                continue;
            for (int i = 0; i < t.stages; ++i, ++at_stage) {
                stage_free(S::kUStages);
                if (!alive)
                    break;
                const int first = t.rows.begin + i * kOuterRows, stage = at_stage % S::kUStages;
                const uint32_t bytes = static_cast<uint32_t>(min(kOuterRows, t.rows.end - first)) * a.rank * 4;
                mbar_arrive_expect_tx(&s_u[stage], bytes);
                bulk_load_g2s(smem + S::kUAt + stage * S::kUBytes,
                              (t.in ? a.dh : a.h) + static_cast<int64_t>(first) * a.rank, bytes, &s_u[stage]);
            }
        }
    } else if (warp == 8) {
        constexpr uint32_t desc = product_desc(128, S::kSide * RP, true, true), first_desc = product_desc(128, RP, true, true);
        constexpr uint32_t next = RP < 64 ? S::kTermBytes : S::kHalfBytes; // the following columns of u's terms
        constexpr uint32_t group = S::kUChunks * 128u;                     // 8 rows of u's terms
        for (int k = 0; k < rounds; ++k) {
            if (!tiles.get(a.rows, k, t) || lane != 0)
                continue;
            for (int i = 0; i < t.stages && alive; ++i, ++at_stage) {
                const int link = i % kOuterChain;
                const int stage = at_stage % S::kStages, u_stage = at_stage % S::kUStages;
                alive = mbar_wait_bounded(&s_v[stage], (at_stage / S::kStages) & 1, a.rows.err) &&
                        mbar_wait_bounded(&s_split[u_stage], (at_stage / S::kUStages) & 1, a.rows.err);
                if (alive && link == 0 && i > 0)
                    alive = mbar_wait_bounded(&s_taken, chains++ & 1, a.rows.err);
                if (!alive)
                    break;
                fence_proxy_async_shared(); // the copies were the other threads'
                tc_fence_after_sync();
                const int steps = (min(kOuterRows, t.rows.end - t.rows.begin - i * kOuterRows) + 15) / 16;
                const uint32_t vs = base + stage * S::kVBytes, us = base + S::kUAt + u_stage * S::kUBytes;
                for (int kk = 0; kk < steps; ++kk) {
                    const uint64_t v = operand_desc(vs + kk * 2048u, Swizzle::k128, S::kHalfBytes, 1024u);
                    const uint32_t from = us + kk * 2 * group;
                    if (S::kSide < 3)
                        tc_product(tmem, v, operand_desc(from, S::kSwizzle, next, group), first_desc, link > 0 || kk > 0);
                    tc_product(tmem + (3 - S::kSide) * RP, v,
                               operand_desc(from + (3 - S::kSide) * S::kTermBytes, S::kSwizzle, next, group), desc,
                               link > 0 || kk > 0);
                }
                tc_commit(&s_free[stage]);
                if (i == t.stages - 1 || link == kOuterChain - 1)
                    tc_commit(&s_done);
            }
        }
    } else {
        constexpr int kVecs = RP / 16; // pieces of 8 ranks a thread and stage
        const int st = tid - 128;
        const uint32_t here = tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16);
        const auto chain_done = [&] {
            if (alive)
                alive = mbar_wait_bounded(&s_done, chains & 1, a.rows.err);
            ++chains;
            tc_fence_after_sync();
        };
        // 16 ranks' sums from j0 on: the terms' of the chain that is done, smallest
        // first, and those of the chains before
        const auto load_sums = [&](float (&v)[16], int j0, bool before) {
            float d[16];
            tmem_load16(v, here + 2 * RP + j0);
            tmem_load16(d, here + RP + j0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] += d[i];
            tmem_load16(d, here + j0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] += d[i];
            if (before) {
                tmem_load16(d, here + 3 * RP + j0);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] += d[i];
            }
        };
        for (int k = 0; k < rounds; ++k) {
            if (!tiles.get(a.rows, k, t))
                continue;
            bool bad = false; // a row of the group has no data
            if (a.rows.row_token != nullptr && t.stages > 0) {
#pragma unroll 4
                for (int row = t.rows.begin + st; row < t.rows.end; row += 128) {
                    const int token = __ldg(a.rows.row_token + row);
                    bad = bad || token < 0 || token >= a.rows.T;
                }
                bad = split_warps_any(bad);
            }
            for (int i = 0; i < t.stages; ++i, ++at_stage) {
                const int stage = at_stage % S::kUStages;
                if (alive)
                    alive = mbar_wait_bounded(&s_u[stage], (at_stage / S::kUStages) & 1, a.rows.err);
                uint8_t* us = smem + S::kUAt + stage * S::kUBytes;
                float4 f[kVecs][2];
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int p = st + j * 128, row = p / (RP / 8), c = p % (RP / 8);
                    const float4* from = reinterpret_cast<const float4*>(us + (row * a.rank + c * 8) * 4);
                    f[j][0] = f[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (c * 8 < a.rank) {
                        f[j][0] = from[0];
                        f[j][1] = from[1];
                    }
                }
                split_warps_sync(); // u is read before its terms take its place
                const int first = t.rows.begin + i * kOuterRows;
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int p = st + j * 128, row = p / (RP / 8), c = p % (RP / 8);
                    if (first + row >= t.rows.end || (bad && row_at(a.rows, first + row, t.rows.end) < 0))
                        f[j][0] = f[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    const uint32_t place = RP < 64 ? swizzled<S::kUChunks>(row, c) : in_halves(row, c);
                    store_terms(us + place, S::kTermBytes, f[j][0], f[j][1]);
                }
                fence_proxy_async_shared();
                mbar_arrive(&s_split[stage]);
                if (i > 0 && i % kOuterChain == 0) { // the chain before, while the next one's first stage is on its way
                    chain_done();
#pragma unroll 1
                    for (int j0 = 0; j0 < RP; j0 += 16) {
                        float v[16];
                        load_sums(v, j0, i > kOuterChain);
                        tmem_store16(here + 3 * RP + j0, v);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s_taken);
                }
            }
            const bool before = t.stages > kOuterChain; // the rows made several chains
            if (t.stages > 0)
                chain_done();
            if (SPLIT) { // this part's sums, where the stages were
#pragma unroll
                for (int j0 = 0; j0 < RP; j0 += 16) {
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = 0.0f;
                    if (t.stages > 0)
                        load_sums(v, j0, before);
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(smem + (st * S::kPitch + j0 + i) * 4) =
                            make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
                tc_fence_before_sync();
                break; // a cluster has one tile
            }
            // thread: column n0 + st, every rank
            const int N = t.in ? a.hidden_in : a.hidden_out, col = t.n0 + st;
            uint16_t* out = static_cast<uint16_t*>(t.in ? a.da : a.db) + static_cast<int64_t>(t.e) * a.rank * N;
#pragma unroll
            for (int j0 = 0; j0 < RP; j0 += 16) {
                if (j0 >= a.rank)
                    break;
                uint32_t d[8]; // two ranks each
                if (t.stages > 0) {
                    float v[16];
                    load_sums(v, j0, before);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[i] = 0u;
                }
                if (col >= N)
                    continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (j0 + 8 * h >= a.rank)
                        break;
                    if (t.in) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            out[static_cast<int64_t>(j0 + 8 * h + i) * N + col] =
                                static_cast<uint16_t>(d[4 * h + i / 2] >> (16 * (i & 1)));
                    } else {
                        st_v4(out + static_cast<int64_t>(col) * a.rank + j0 + 8 * h,
                              make_uint4(d[4 * h], d[4 * h + 1], d[4 * h + 2], d[4 * h + 3]));
                    }
                }
            }
            tc_fence_before_sync(); // the next tile's first product follows the splits of its first stage
        }
    }
    __syncthreads();
    if (warp == 8)
        tmem_free(tmem, S::kTmem);
    if (SPLIT && tiles.get(a.rows, 0, t)) { // the parts' sums, in their order; a part has its share of the columns
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int N = t.in ? a.hidden_in : a.hidden_out;
        const int share = (kOuterCols + parts - 1) / parts, c0 = tiles.part * share, cols = min(share, kOuterCols - c0);
        uint16_t* out = static_cast<uint16_t*>(t.in ? a.da : a.db) + static_cast<int64_t>(t.e) * a.rank * N;
        for (int i = tid; i < cols * (a.rank / 8); i += kOuterThreads) {
            const int c = c0 + i % cols, j = i / cols * 8, col = t.n0 + c;
            float4 v[kOuterParts][2]; // all on their way at once
#pragma unroll
            for (int p = 0; p < kOuterParts; ++p) {
                const float4* from = reinterpret_cast<const float4*>(
                    cluster.map_shared_rank(smem, min(p, parts - 1)) + (c * S::kPitch + j) * 4);
                v[p][0] = from[0];
                v[p][1] = from[1];
            }
            float4 s0 = v[0][0], s1 = v[0][1];
#pragma unroll
            for (int p = 1; p < kOuterParts; ++p)
                if (p < parts) {
                    s0 = make_float4(s0.x + v[p][0].x, s0.y + v[p][0].y, s0.z + v[p][0].z, s0.w + v[p][0].w);
                    s1 = make_float4(s1.x + v[p][1].x, s1.y + v[p][1].y, s1.z + v[p][1].z, s1.w + v[p][1].w);
                }
            if (col >= N)
                continue;
            const uint32_t d[4] = {pack_bf16x2(s0.x, s0.y), pack_bf16x2(s0.z, s0.w), pack_bf16x2(s1.x, s1.y),
                                   pack_bf16x2(s1.z, s1.w)};
            if (t.in) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    out[static_cast<int64_t>(j + k) * N + col] = static_cast<uint16_t>(d[k / 2] >> (16 * (k & 1)));
            } else {
                st_v4(out + static_cast<int64_t>(col) * a.rank + j, make_uint4(d[0], d[1], d[2], d[3]));
            }
        }
        cluster.sync(); // no CTA leaves while its sums are read
    }
}

// -------------------------------------------------------------- row tokens
__global__ void __launch_bounds__(256) row_tokens_kernel(RowTokensLaunch a)
{
    const int64_t p = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (p >= static_cast<int64_t>(a.T) * a.rows.K)
        return;
    const int s = __ldg(a.rows.slot + p);
    const int64_t e = __ldg(a.rows.topk_idx + p);
    if (s < 0 || e < 0 || e >= a.rows.E)
        return;
    int64_t row = s;
    if (a.rows.mode == EP_LAYOUT_COMPACT) {
        row += __ldg(a.rows.offsets + e);
    } else if (s < a.rows.max_tokens) {
        row += e * a.rows.max_tokens;
    } else {
        flag_error(a.err, EP_DEVERR_OVERFLOW);
        return;
    }
    if (row < 0 || row >= a.rows.num_rows) {
        flag_error(a.err, EP_DEVERR_OVERFLOW);
        return;
    }
    a.row_token[row] = static_cast<int32_t>(p / a.rows.K);
}

// ---------------------------------------------------------------- launches
// Calls f with the smallest padded rank (16, 32, 64, 128) that holds `rank`.
template <typename F>
cudaError_t with_rank(int rank, F&& f)
{
    if (rank <= 16)
        return f(std::integral_constant<int, 16>{});
    if (rank <= 32)
        return f(std::integral_constant<int, 32>{});
    if (rank <= 64)
        return f(std::integral_constant<int, 64>{});
    return f(std::integral_constant<int, 128>{});
}

// A launch as a programmatic dependent, in clusters of `cluster`: every kernel
// here waits (pdl_wait) before it reads what the kernel before may have written.
template <auto KERNEL, typename... Args>
cudaError_t launch_after(unsigned grid, unsigned block, int smem, int cluster, cudaStream_t stream, const Args&... args)
{
    // the devices on which the kernel may use its shared memory already (host
    // threads may race to set a bit; they set the same attribute)
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (smem > 48 * 1024 && (ready.load(std::memory_order_relaxed) & bit) == 0) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
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
    return cudaLaunchKernelEx(&cfg, KERNEL, args...);
}

} // namespace

cudaError_t launch_row_tokens(const RowTokensLaunch& a, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    if (a.rows.num_rows > 0)
        e = cudaMemsetAsync(a.row_token, 0xff, static_cast<size_t>(a.rows.num_rows) * 4, stream);
    const int64_t pairs = static_cast<int64_t>(a.T) * a.rows.K;
    if (e != cudaSuccess || pairs == 0)
        return e;
    row_tokens_kernel<<<static_cast<unsigned>((pairs + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_lora_shrink(const LoraShrinkLaunch& a, cudaStream_t stream)
{
    if (a.rows.pairs == 0)
        return cudaSuccess;
    if (a.rows.num_rows == 0)
        return launch_after<overflow_kernel>(1, 32, 0, 1, stream, a.rows);
    const int tiles = most_tiles(a.rows, kShrinkTile);
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        using S = ShrinkShape<RP>;
        CUtensorMap w_map;
        const cudaError_t st = a.transposed ? encode_map(&w_map, a.w, a.rank, a.K, a.rows.E, S::kWBox, kDepth)
                                            : encode_map(&w_map, a.w, a.K, a.rank, a.rows.E, 64, RP);
        if (st != cudaSuccess)
            return st;
        const int steps = (a.K + kDepth - 1) / kDepth;
        // One resident wave of clusters: forward of 4096 rows of 16 adapters 51 us,
        // with room for 444 CTAs 58 us (the last clusters wait for free places).
        const int parts = std::max(1, std::min({8, 2 * 148 / tiles, steps / 4}));
        const unsigned grid = static_cast<unsigned>(tiles) * parts;
        return a.transposed ? launch_after<lora_shrink_kernel<RP, true>>(grid, S::kThreads, S::kBytes, parts, stream, w_map, a)
                            : launch_after<lora_shrink_kernel<RP, false>>(grid, S::kThreads, S::kBytes, parts, stream, w_map, a);
    });
}

cudaError_t launch_lora_expand(const LoraExpandLaunch& a, cudaStream_t stream)
{
    const int tiles = most_tiles(a.rows, kExpandTile);
    const int steps = (a.N + kExpandCols - 1) / kExpandCols;
    const int shares = static_cast<int>(
        std::min<int64_t>(static_cast<int64_t>(tiles) * steps, std::max(kExpandGrid, tiles)));
    const int64_t grid = shares + (a.slot != nullptr ? (a.rows.T + kRowTile - 1) / kRowTile : 0);
    if (grid == 0)
        return cudaSuccess;
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        using S = ExpandShape<RP>;
        CUtensorMap w_map;
        const cudaError_t e = a.transposed ? encode_map(&w_map, a.w, a.N, a.rank, a.rows.E, 64, RP)
                                           : encode_map(&w_map, a.w, a.rank, a.N, a.rows.E, S::kBox, kExpandCols);
        if (e != cudaSuccess)
            return e;
        const unsigned ctas = static_cast<unsigned>(grid);
        return a.transposed
                   ? launch_after<lora_expand_kernel<RP, true>>(ctas, kExpandThreads, S::kBytes, 1, stream, w_map, a, shares)
                   : launch_after<lora_expand_kernel<RP, false>>(ctas, kExpandThreads, S::kBytes, 1, stream, w_map, a, shares);
    });
}

// Is a forward call one for lora_few_kernel: by the rows an adapter has on
// average, the fewer the more ranks its registers have to hold, or by all rows,
// where the other kernels' starts and ends weigh more.  Measured at 4096 -> 4096
// against the kernels for many rows, us:
//   rank 16: 16 rows 7.4 / 16.4 and 10.6 / 29 (16, 64 adapters), 256 rows 24 / 30
//   rank 32: 16 rows 9.2 / 17.0, 64 rows 35 / 41 (64 adapters), 256 rows 33.6 / 33.0
//   rank 64: 16 rows 13.0 / 18.4 and 28 / 35, 64 rows 25.1 / 20.7 and 54 / 47
//   one adapter, rank 16: 1024 rows 10.4 / 17.3, 4096 rows 25.1 / 27.9
//   8 adapters, rank 32: 768 rows 12.9 / 17.4, 2048 rows 19.6 / 22.0
//   one adapter, rank 64: 128 rows 10.2 / 11.3, 256 rows 13.0 / 12.0
// The adapters in memory are counted, since the host does not know which have rows.
// All rows with one of many: rank 16 4096 rows of 256 adapters 26 / 39, 16384 of 1024
// 214 / 286; rank 32 35 / 41 and 233 / 290; rank 64 1024 rows of 64 25.8 / 21.7, 4096 of
// 256 56 / 44, 16384 of 1024 299 / 315.
bool lora_few(const LoraRows& rows, int rank)
{
    if (rank > kFewRank || rows.pairs == 0 || rows.num_rows == 0)
        return false;
    const int64_t each = rank <= 16 ? 256 : (rank <= 32 ? 64 : 16), all = rank <= 32 ? 2048 : 128;
    return rows.pairs <= std::max(each * rows.E, all);
}

cudaError_t launch_lora_few(const LoraFewLaunch& a, cudaStream_t stream)
{
    const int tiles = most_tiles(a.rows, kFewTile);
    const int parts = std::max(1, std::min(kFewCluster, 2 * 148 / tiles)); // one resident wave
    const int copies = a.slot != nullptr ? (a.rows.T + kRowTile - 1) / kRowTile : 0;
    const unsigned grid = static_cast<unsigned>(tiles + (copies + parts - 1) / parts) * parts;
    const auto run = [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        return launch_after<lora_few_kernel<RP>>(grid, kFewThreads, FewShape<RP>::kBytes, parts, stream, a, tiles);
    };
    if (a.rank <= 16)
        return run(std::integral_constant<int, 16>{});
    if (a.rank <= 32)
        return run(std::integral_constant<int, 32>{});
    return run(std::integral_constant<int, kFewRank>{});
}

cudaError_t launch_lora_outer(const LoraOuterLaunch& a, cudaStream_t stream)
{
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        using S = OuterShape<RP>;
        const int in_tiles = (a.hidden_in + kOuterCols - 1) / kOuterCols;
        const int out_tiles = (a.hidden_out + kOuterCols - 1) / kOuterCols;
        const int64_t total = static_cast<int64_t>(a.rows.E) * (in_tiles + out_tiles);
        // Fewer tiles than places (one adapter, narrow layers): parts of kPartStages
        // stages and more.  4096 rows of one adapter, rank 64, 4096 -> 4096: all
        // gradients 67 us, whole tiles 108; 1024 rows, rank 32, 7168 -> 7168: in two
        // parts 36.9 us, whole 35.8 (a cluster starts later and joins).
        constexpr int kPartStages = 8;
        const int64_t places = 148 * S::kCtas, stages = a.rows.pairs / a.rows.E / kOuterRows;
        const int parts = static_cast<int>(std::max<int64_t>(
            1, std::min({static_cast<int64_t>(kOuterParts), places / total, stages / kPartStages})));
        if (parts > 1)
            return launch_after<lora_outer_kernel<RP, true>>(static_cast<unsigned>(total * parts), kOuterThreads, S::kBytes,
                                                             parts, stream, a, in_tiles, out_tiles, parts);
        return launch_after<lora_outer_kernel<RP, false>>(static_cast<unsigned>(std::min(total, places)), kOuterThreads,
                                                          S::kBytes, 1, stream, a, in_tiles, out_tiles, 1);
    });
}

} // namespace ep
