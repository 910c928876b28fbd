// ep_lora.cu -- low-rank adapters on the rows of a token-choice layout.
//
// The layout groups rows by adapter, so a tile of kRowTile rows of one group is
// an ordinary matrix product with that adapter's factors: the rows are read
// where they are (row_token, or the dispatched rows themselves).  Three
// products, all memory-bound at the ranks they are for (rank flops a byte of
// row data):
//   shrink  u = s_e X W        long sum over the hidden width, rank columns
//   expand  out = base + u W   rank-long sum, hidden columns, base and out move
//   outer   dW = sum of rows   sum over a group's rows
// Tensor-core products of bf16 operands with fp32 sums; u (fp32) enters as
// hi + lo (ep_mma.cuh).
#include <algorithm>

#include <cooperative_groups.h>

#include "ep_lora_launch.h"
#include "ep_mma.cuh"
#include "ep_tcgen05.cuh"

namespace ep {

namespace cg = cooperative_groups;

namespace {

constexpr int kRowTile = 64;

// ------------------------------------------------------------------- rows
struct RowRange {
    int begin, end;
};

// Rows of adapter e, within [0, num_rows).
__device__ __forceinline__ RowRange group_rows(const LoraRows& g, int e)
{
    int64_t b, n;
    if (g.mode == EP_LAYOUT_COMPACT) {
        b = __ldg(g.offsets + e);
        n = __ldg(g.offsets + e + 1) - b;
    } else {
        b = static_cast<int64_t>(e) * g.max_tokens;
        n = min(__ldg(g.counts + e), g.max_tokens);
    }
    b = min(max(b, int64_t{0}), static_cast<int64_t>(g.num_rows));
    n = min(max(n, int64_t{0}), static_cast<int64_t>(g.num_rows) - b);
    return {static_cast<int>(b), static_cast<int>(b + n)};
}

// Tiles of kRowTile rows are numbered adapter after adapter: the adapter and rows of
// tile i; false when there are fewer.  One warp; all lanes get the answer.
__device__ __forceinline__ bool find_tile(const LoraRows& g, int i, int lane, int& e, RowRange& rows)
{
    const int per = (g.E + 31) / 32; // adapters a lane, consecutive
    const int e0 = min(lane * per, g.E), e1 = min(e0 + per, g.E);
    int n = 0;
#pragma unroll 8
    for (int j = e0; j < e1; ++j) {
        const RowRange r = group_rows(g, j);
        n += (r.end - r.begin + kRowTile - 1) / kRowTile;
    }
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFullMask, inc, d);
        if (lane >= d)
            inc += o;
    }
    const uint32_t past = __ballot_sync(kFullMask, inc > i);
    if (past == 0u)
        return false;
    const int from = __ffs(past) - 1;
    int found = 0, b = 0, end = 0;
    if (lane == from) {
        int left = i - (inc - n);
        for (int j = e0; j < e1; ++j) {
            const RowRange r = group_rows(g, j);
            const int tiles = (r.end - r.begin + kRowTile - 1) / kRowTile;
            if (left < tiles) {
                found = j;
                b = r.begin + left * kRowTile;
                end = min(r.end, b + kRowTile);
                break;
            }
            left -= tiles;
        }
    }
    e = __shfl_sync(kFullMask, found, from);
    rows.begin = __shfl_sync(kFullMask, b, from);
    rows.end = __shfl_sync(kFullMask, end, from);
    return true;
}

// Rows that the routing fills past num_rows are left out; the first CTA of a
// call's first kernel says so.  One warp.
__device__ __forceinline__ void report_overflow(const LoraRows& g, int lane)
{
    bool over = false;
    for (int e = lane; e < g.E; e += 32) {
        const int64_t end = g.mode == EP_LAYOUT_COMPACT ? static_cast<int64_t>(__ldg(g.offsets + e + 1))
                                                        : static_cast<int64_t>(e) * g.max_tokens + __ldg(g.counts + e);
        const bool full = g.mode != EP_LAYOUT_COMPACT && __ldg(g.counts + e) > g.max_tokens;
        over = over || full || (end > g.num_rows && (g.mode == EP_LAYOUT_COMPACT || __ldg(g.counts + e) > 0));
    }
    if (over)
        flag_error(g.err, EP_DEVERR_OVERFLOW);
}

// Most tiles that the rows can make: a full one for every kRowTile rows and a part
// one for every adapter in use.
int most_tiles(const LoraRows& g)
{
    const int rows = std::min(g.pairs, g.num_rows);
    return rows / kRowTile + std::min(g.E, rows);
}

// Where the data of `row` is: its row index in x, base or out; -1 when the
// row is past the group's end or its token is out of range.
__device__ __forceinline__ int row_at(const LoraRows& g, int row, int end)
{
    if (row >= end)
        return -1;
    if (g.row_token == nullptr)
        return row;
    const int t = __ldg(g.row_token + row);
    if (t < 0 || t >= g.T) {
        flag_error(g.err, EP_DEVERR_BAD_INDEX);
        return -1;
    }
    return t;
}

// ------------------------------------------------------------------ shrink
constexpr int kShrinkThreads = 128; // four warps, 16 rows each
constexpr int kDepth = 64;          // hidden channels a stage

template <int RP>
struct ShrinkShape {
    static constexpr int kStages = RP <= 64 ? 4 : 3;
    static constexpr int kXBytes = kRowTile * kDepth * 2;
    static constexpr int kWBytes = RP * kDepth * 2;
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kPitch = RP + 4; // floats a row of the partial sums
    static constexpr int kSumBytes = kRowTile * kPitch * 4;
    static constexpr int kBytes = kStages * kStageBytes > kSumBytes ? kStages * kStageBytes : kSumBytes;
};

// A cluster has one tile of rows; its CTAs split the hidden width, and each
// adds up its share of the tile's rows over the cluster, in CTA order (the
// same sum every time, no atomics, no partial sums in HBM).
template <int RP, bool TRANS>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(LoraShrinkLaunch a)
{
    using S = ShrinkShape<RP>;
    extern __shared__ __align__(128) uint8_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && warp == 0)
        report_overflow(a.rows, lane);
    int e;
    RowRange rows;
    if (!find_tile(a.rows, blockIdx.x / parts, lane, e, rows))
        return; // the whole cluster has the same tile
    const int steps = (a.K + kDepth - 1) / kDepth;
    const int per = (steps + parts - 1) / parts;
    const int s0 = min(part * per, steps), n = min(per, steps - s0);
    const uint32_t base = smem_addr(smem);

    // this thread's copies: chunk tid % 8 of rows tid / 8 + 16 i of x
    const uint16_t* x_row[4];
    bool x_on[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = row_at(a.rows, rows.begin + tid / 8 + 16 * i, rows.end);
        x_on[i] = at >= 0;
        x_row[i] = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(max(at, 0)) * a.K;
    }
    const uint16_t* w = static_cast<const uint16_t*>(a.w) + static_cast<int64_t>(e) * a.rank * a.K;

    const auto load = [&](int step, int stage) {
        const uint32_t xs = base + stage * S::kStageBytes, ws = xs + S::kXBytes;
        const int k0 = step * kDepth;
        const int c = tid % 8, k = k0 + c * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            cp_async16(xs + swizzled<8>(tid / 8 + 16 * i, c), x_row[i] + (k < a.K ? k : 0),
                       x_on[i] && k < a.K ? 16 : 0);
        if (!TRANS) {
#pragma unroll
            for (int j = tid / 8; j < RP; j += 16) {
                const bool on = j < a.rank && k < a.K;
                cp_async16(ws + swizzled<8>(j, c), on ? w + static_cast<int64_t>(j) * a.K + k : w, on ? 16 : 0);
            }
        } else {
            constexpr int PC = RP / 8;
#pragma unroll
            for (int i = tid; i < kDepth * PC; i += kShrinkThreads) {
                const int row = i / PC, cc = i % PC;
                const bool on = cc * 8 < a.rank && k0 + row < a.K;
                cp_async16(ws + swizzled<PC>(row, cc), on ? w + static_cast<int64_t>(k0 + row) * a.rank + cc * 8 : w,
                           on ? 16 : 0);
            }
        }
    };

    float acc[RP / 8][4];
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[j][i] = 0.0f;
    const bool busy = rows.begin + warp * 16 < rows.end; // this warp has rows

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
        if (i < n)
            load(s0 + i, i);
        cp_async_commit();
    }
    for (int i = 0; i < n; ++i) {
        cp_async_wait<S::kStages - 2>();
        __syncthreads();
        if (i + S::kStages - 1 < n)
            load(s0 + i + S::kStages - 1, (i + S::kStages - 1) % S::kStages);
        cp_async_commit();
        if (!busy)
            continue;
        const uint32_t xs = base + (i % S::kStages) * S::kStageBytes, ws = xs + S::kXBytes;
#pragma unroll
        for (int kk = 0; kk < kDepth / 16; ++kk) {
            uint32_t x4[4];
            ldmatrix4(x4, xs + swizzled<8>(warp * 16 + (lane & 15), kk * 2 + (lane >> 4)));
#pragma unroll
            for (int j = 0; j < RP / 16; ++j) {
                uint32_t b[4];
                if (!TRANS)
                    ldmatrix4(b, ws + swizzled<8>(j * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
                else
                    ldmatrix4_trans(b, ws + swizzled<RP / 8>(kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3),
                                                             j * 2 + (lane >> 4)));
                mma16816(acc[2 * j], x4, b[0], b[1]);
                mma16816(acc[2 * j + 1], x4, b[2], b[3]);
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // the tile's partial sums to shared memory, then the cluster's sums of them
    float* sums = reinterpret_cast<float*>(smem);
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int j = 0; j < RP / 8; ++j) {
        float* p = sums + (warp * 16 + g) * S::kPitch + j * 8 + 2 * q;
        *reinterpret_cast<float2*>(p) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(p + 8 * S::kPitch) = make_float2(acc[j][2], acc[j][3]);
    }
    cluster.sync();
    const float scale = a.scales != nullptr ? __ldg(a.scales + e) : 1.0f;
    const int vecs = a.rank / 4;
    const int live = rows.end - rows.begin;
    for (int i = part * kShrinkThreads + tid; i < live * vecs; i += parts * kShrinkThreads) {
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
constexpr int kExpandThreads = 256; // warps: 4 of 16 rows x 2 of 128 columns
constexpr int kColTile = 256;

// Word i of lane q of each quad <-> word q of lane i.
__device__ __forceinline__ void transpose_quad(uint32_t (&w)[4], int q)
{
    const bool up2 = (q & 2) != 0, up1 = (q & 1) != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t r = __shfl_xor_sync(kFullMask, up2 ? w[i] : w[i + 2], 2);
        if (up2)
            w[i] = r;
        else
            w[i + 2] = r;
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t r = __shfl_xor_sync(kFullMask, up1 ? w[i] : w[i + 1], 1);
        if (up1)
            w[i] = r;
        else
            w[i + 1] = r;
    }
}

__device__ __forceinline__ uint32_t add_to_bf16x2(uint32_t base, float a, float b)
{
    return pack_bf16x2(bf16_lo(base) + a, bf16_hi(base) + b);
}

// Each thread ends with 8 consecutive columns of a row (one 16-byte load and
// store): for w [N, rank] the columns of w's tile are laid out in shared memory
// in the order in which the product's fragments hand them out; for w [rank, N]
// the quad's four lanes exchange words.
template <int RP, bool TRANS>
__global__ void __launch_bounds__(kExpandThreads, RP <= 64 ? 2 : 1) lora_expand_kernel(LoraExpandLaunch a, int tiles,
                                                                                         int col_tiles)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = blockIdx.x / col_tiles;
    if (blockIdx.x >= static_cast<unsigned>(tiles) * col_tiles) { // tokens without an adapter: out = base
        const int t0 = (blockIdx.x - tiles * col_tiles) * kRowTile;
        for (int i = warp; i < kRowTile; i += kExpandThreads / 32) {
            const int t = t0 + i;
            if (t >= a.rows.T || __ldg(a.slot + t) >= 0)
                continue;
            const int64_t at = static_cast<int64_t>(t) * a.N;
            for (int c = lane * 8; c < a.N; c += 256) {
                const uint4 v = a.base != nullptr ? ld_nc_v4(static_cast<const uint16_t*>(a.base) + at + c)
                                                  : make_uint4(0u, 0u, 0u, 0u);
                st_v4(static_cast<uint16_t*>(a.out) + at + c, v);
            }
        }
        return;
    }
    int e;
    RowRange rows;
    if (!find_tile(a.rows, tile, lane, e, rows))
        return;
    const int n0 = (blockIdx.x - tile * col_tiles) * kColTile;
    const uint32_t ws = smem_addr(smem);
    const uint16_t* w = static_cast<const uint16_t*>(a.w) + static_cast<int64_t>(e) * a.rank * a.N;
    constexpr int PC = RP / 8;
    if (!TRANS) {
#pragma unroll 4
        for (int i = tid; i < kColTile * PC; i += kExpandThreads) {
            const int col = i / PC, c = i % PC;
            // column 8a + 2j + b of 32 at place 8j + 2a + b
            const int place = (col & ~31) | ((col & 6) << 2) | ((col & 24) >> 2) | (col & 1);
            const bool on = c * 8 < a.rank && n0 + col < a.N;
            cp_async16(ws + swizzled<PC>(place, c), on ? w + static_cast<int64_t>(n0 + col) * a.rank + c * 8 : w,
                       on ? 16 : 0);
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < RP * (kColTile / 8); i += kExpandThreads) {
            const int row = i / (kColTile / 8), c = i % (kColTile / 8);
            const bool on = row < a.rank && n0 + c * 8 < a.N;
            cp_async16(ws + swizzled<kColTile / 8>(row, c), on ? w + static_cast<int64_t>(row) * a.N + n0 + c * 8 : w,
                       on ? 16 : 0);
        }
    }
    cp_async_commit();

    const int g = lane >> 2, q = lane & 3;
    const int wm = warp & 3, wn = warp >> 2; // rows 16 wm.., columns 128 wn..
    const int row0 = rows.begin + wm * 16 + g;
    const int at0 = row_at(a.rows, row0, rows.end), at1 = row_at(a.rows, row0 + 8, rows.end);
    const int64_t o0 = static_cast<int64_t>(max(at0, 0)) * a.N, o1 = static_cast<int64_t>(max(at1, 0)) * a.N;
    // base, all of it at once: 4 x 32 columns of two rows
    uint4 base[4][2];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int col = n0 + wn * 128 + c * 32 + q * 8;
        const bool on = a.base != nullptr && col < a.N;
        const uint16_t* b = static_cast<const uint16_t*>(a.base);
        base[c][0] = on && at0 >= 0 ? ld_nc_v4(b + o0 + col) : make_uint4(0u, 0u, 0u, 0u);
        base[c][1] = on && at1 >= 0 ? ld_nc_v4(b + o1 + col) : make_uint4(0u, 0u, 0u, 0u);
    }
    // u of this thread's rows, in two terms
    uint32_t hi[RP / 16][4], lo[RP / 16][4];
    const float* u0 = a.u + static_cast<int64_t>(row0) * a.rank;
    const float* u1 = u0 + static_cast<int64_t>(8) * a.rank;
#pragma unroll
    for (int ks = 0; ks < RP / 16; ++ks) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = ks * 16 + h * 8 + 2 * q;
            const float2 zero = make_float2(0.0f, 0.0f);
            const float2 v0 = at0 >= 0 && j < a.rank ? __ldcg(reinterpret_cast<const float2*>(u0 + j)) : zero;
            const float2 v1 = at1 >= 0 && j < a.rank ? __ldcg(reinterpret_cast<const float2*>(u1 + j)) : zero;
            split_bf16x2(v0.x, v0.y, hi[ks][2 * h], lo[ks][2 * h]);
            split_bf16x2(v1.x, v1.y, hi[ks][2 * h + 1], lo[ks][2 * h + 1]);
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    if (rows.begin + wm * 16 >= rows.end)
        return; // no rows in this warp

#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[j][i] = 0.0f;
        const int place = wn * 128 + c * 32;
#pragma unroll
        for (int ks = 0; ks < RP / 16; ++ks) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                uint32_t b[4];
                if (!TRANS)
                    ldmatrix4(b, ws + swizzled<PC>(place + j * 8 + (lane & 7) + ((lane >> 4) << 3),
                                                   ks * 2 + ((lane >> 3) & 1)));
                else
                    ldmatrix4_trans(b, ws + swizzled<kColTile / 8>(ks * 16 + (lane & 7) + (((lane >> 3) & 1) << 3),
                                                                   place / 8 + j + (lane >> 4)));
                mma16816(acc[j], hi[ks], b[0], b[1]);
                mma16816(acc[j + 1], hi[ks], b[2], b[3]);
                mma16816(acc[j], lo[ks], b[0], b[1]);
                mma16816(acc[j + 1], lo[ks], b[2], b[3]);
            }
        }
        const int col = n0 + place + q * 8;
        uint16_t* out = static_cast<uint16_t*>(a.out);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t v[4] = {base[c][r].x, base[c][r].y, base[c][r].z, base[c][r].w};
            if (TRANS)
                transpose_quad(v, q);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = add_to_bf16x2(v[j], acc[j][2 * r], acc[j][2 * r + 1]);
            if (TRANS)
                transpose_quad(v, q);
            if ((r == 0 ? at0 : at1) >= 0 && col < a.N)
                st_v4(out + (r == 0 ? o0 : o1) + col, make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
}

// ------------------------------------------------------------------- outer
// dW of one adapter and 128 columns of x or dy: the columns are the product's
// rows (M), the rank its columns (N), and the sum runs over the adapter's rows,
// 64 at a time.  Both operands are MN-major: the row data as it lies in HBM,
// and u, which the threads write as two bf16 tiles (hi, lo).  Sums stay in
// tensor memory until the last row.
constexpr int kOuterThreads = 128;
constexpr int kOuterCols = 128;
constexpr int kOuterStages = 4;
constexpr int kOuterAhead = kOuterStages - 2; // chunks in flight while one is multiplied

template <int RP>
struct OuterShape {
    static constexpr int kVBytes = kRowTile * kOuterCols * 2;
    static constexpr int kUBytes = kRowTile * RP * 2; // one term
    static constexpr int kStageBytes = kVBytes + 2 * kUBytes;
    static constexpr int kBytes = kOuterStages * kStageBytes + 1024; // tiles start on 1024 bytes
    static constexpr int kCols = RP < 32 ? 32 : RP;                  // tensor memory
    static constexpr Swizzle kSwizzle = RP == 16 ? Swizzle::k32 : (RP == 32 ? Swizzle::k64 : Swizzle::k128);
    static constexpr int kUChunks = RP < 64 ? RP / 8 : 8; // 16-byte chunks a row of u's tile
};

// Place of columns 8c.. of `row` in a tile of 128-byte rows, 64 columns each.
__device__ __forceinline__ uint32_t halves(int row, int c)
{
    return static_cast<uint32_t>(c >> 3) * (kRowTile * 128u) + swizzled<8>(row, c & 7);
}

template <int RP>
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(LoraOuterLaunch a, int in_tiles, int out_tiles)
{
    using S = OuterShape<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_free[kOuterStages], s_done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_at[2][kRowTile];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int per = in_tiles + out_tiles;
    const int e = blockIdx.x / per, i_tile = blockIdx.x - e * per;
    const bool in = i_tile < in_tiles; // da, from x and dh; else db, from dy and h
    const int N = in ? a.hidden_in : a.hidden_out;
    const int n0 = (in ? i_tile : i_tile - in_tiles) * kOuterCols;
    const uint16_t* v = static_cast<const uint16_t*>(in ? a.x : a.dy);
    const float* u = in ? a.dh : a.h;
    const RowRange rows = group_rows(a.rows, e);
    const int n = (rows.end - rows.begin + kRowTile - 1) / kRowTile;
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_addr(smem);

    uint32_t tmem = 0;
    if (n > 0) {
        if (warp == 0)
            tmem_alloc(&s_tmem, S::kCols);
        if (tid == 0) {
            for (int i = 0; i < kOuterStages; ++i)
                mbar_init(&s_free[i], 1);
            mbar_init(&s_done, 1);
            fence_mbar_init();
        }
        // where the rows' data is: of chunk i in s_at[i % 2], of the one after in a register
        const auto at_of = [&](int chunk) {
            return tid < kRowTile ? row_at(a.rows, rows.begin + chunk * kRowTile + tid, rows.end) : -1;
        };
        if (tid < kRowTile)
            s_at[0][tid] = at_of(0);
        int next_at = at_of(1);
        // u of the next chunk, in registers
        constexpr int kVecs = RP / 16;
        float4 un[kVecs][2];
        const auto load_u = [&](int chunk) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int t = tid + i * kOuterThreads, row = rows.begin + chunk * kRowTile + t / (RP / 8), c = t % (RP / 8);
                un[i][0] = un[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (row < rows.end && c * 8 < a.rank) {
                    const float4* p = reinterpret_cast<const float4*>(u + static_cast<int64_t>(row) * a.rank + c * 8);
                    un[i][0] = __ldcg(p);
                    un[i][1] = __ldcg(p + 1);
                }
            }
        };
        load_u(0);
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        tmem = s_tmem;

        bool alive = true; // false once a wait has run out
        for (int it = 0; it < n + kOuterAhead; ++it) {
            if (it < n) {
                const int stage = it % kOuterStages;
                if (it >= kOuterStages && alive)
                    alive = mbar_wait_bounded(&s_free[stage], (it / kOuterStages - 1) & 1, a.rows.err);
                const uint32_t vs = base + stage * S::kStageBytes;
                const int* at = s_at[it & 1];
                const int c = tid % 16, col = n0 + c * 8;
#pragma unroll
                for (int i = 0; i < kRowTile / 8; ++i) {
                    const int row = tid / 16 + 8 * i, r = at[row];
                    const bool on = r >= 0 && col < N;
                    cp_async16(vs + halves(row, c), on ? v + static_cast<int64_t>(r) * N + col : v, on ? 16 : 0);
                }
                uint8_t* us = smem + stage * S::kStageBytes + S::kVBytes;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int t = tid + i * kOuterThreads, row = t / (RP / 8), cu = t % (RP / 8);
                    uint4 h4 = make_uint4(0u, 0u, 0u, 0u), l4 = h4;
                    if (at[row] >= 0) {
                        split_bf16x2(un[i][0].x, un[i][0].y, h4.x, l4.x);
                        split_bf16x2(un[i][0].z, un[i][0].w, h4.y, l4.y);
                        split_bf16x2(un[i][1].x, un[i][1].y, h4.z, l4.z);
                        split_bf16x2(un[i][1].z, un[i][1].w, h4.w, l4.w);
                    }
                    const uint32_t place = RP < 64 ? swizzled<S::kUChunks>(row, cu) : halves(row, cu);
                    *reinterpret_cast<uint4*>(us + place) = h4;
                    *reinterpret_cast<uint4*>(us + S::kUBytes + place) = l4;
                }
                load_u(it + 1);
                if (tid < kRowTile)
                    s_at[(it + 1) & 1][tid] = next_at;
                next_at = at_of(it + 2);
            }
            cp_async_commit();
            const int j = it - kOuterAhead;
            cp_async_wait<kOuterAhead>();
            fence_proxy_async_shared();
            __syncthreads();
            if (j >= 0 && tid == 0) {
                tc_fence_after_sync();
                const uint32_t vs = base + (j % kOuterStages) * S::kStageBytes, us = vs + S::kVBytes;
                constexpr uint32_t desc = product_desc(kOuterCols, RP, true, true);
                constexpr uint32_t group = S::kUChunks * 128u; // 8 rows of u
#pragma unroll
                for (int kk = 0; kk < kRowTile / 16; ++kk) {
                    const uint64_t va = operand_desc(vs + kk * 2048u, Swizzle::k128, kRowTile * 128u, 1024u);
                    tc_product(tmem, va, operand_desc(us + kk * 2 * group, S::kSwizzle, kRowTile * 128u, group), desc,
                               j > 0 || kk > 0);
                    tc_product(tmem, va,
                               operand_desc(us + S::kUBytes + kk * 2 * group, S::kSwizzle, kRowTile * 128u, group), desc,
                               true);
                }
                tc_commit(j == n - 1 ? &s_done : &s_free[j % kOuterStages]);
            }
        }
        if (alive)
            mbar_wait_bounded(&s_done, 0, a.rows.err);
        tc_fence_after_sync();
    }

    // thread: column n0 + tid, every rank
    const int col = n0 + tid;
    uint16_t* out = static_cast<uint16_t*>(in ? a.da : a.db) + static_cast<int64_t>(e) * a.rank * N;
#pragma unroll
    for (int j0 = 0; j0 < RP; j0 += 16) {
        if (j0 >= a.rank)
            break;
        float d[16];
        if (n > 0) {
            tmem_load16(d, tmem + (static_cast<uint32_t>(warp * 32) << 16) + j0);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                d[i] = 0.0f;
        }
        if (col < N) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (j0 + 8 * h >= a.rank)
                    break;
                if (in) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        out[static_cast<int64_t>(j0 + 8 * h + i) * N + col] =
                            static_cast<uint16_t>(pack_bf16x2(d[8 * h + i], 0.0f));
                } else {
                    st_v4(out + static_cast<int64_t>(col) * a.rank + j0 + 8 * h,
                          make_uint4(pack_bf16x2(d[8 * h], d[8 * h + 1]), pack_bf16x2(d[8 * h + 2], d[8 * h + 3]),
                                     pack_bf16x2(d[8 * h + 4], d[8 * h + 5]), pack_bf16x2(d[8 * h + 6], d[8 * h + 7])));
                }
            }
        }
    }
    if (n > 0) {
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0)
            tmem_free(tmem, S::kCols);
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

template <typename K>
cudaError_t allow_smem(K kernel, int bytes)
{
    if (bytes <= 48 * 1024)
        return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
    const int tiles = std::max(1, most_tiles(a.rows)); // one at least: it reports rows past the buffer
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        const auto kernel = a.transposed ? lora_shrink_kernel<RP, true> : lora_shrink_kernel<RP, false>;
        const int smem = ShrinkShape<RP>::kBytes;
        cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess)
            return e;
        const int steps = (a.K + kDepth - 1) / kDepth;
        int parts = 1;
        while (parts < 8 && tiles * parts < 3 * 148 && steps >= 8 * parts)
            parts *= 2;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(tiles) * parts);
        cfg.blockDim = dim3(kShrinkThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {static_cast<unsigned>(parts), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, a);
    });
}

cudaError_t launch_lora_expand(const LoraExpandLaunch& a, cudaStream_t stream)
{
    const int tiles = most_tiles(a.rows);
    const int col_tiles = (a.N + kColTile - 1) / kColTile;
    const int64_t grid = static_cast<int64_t>(tiles) * col_tiles +
                         (a.slot != nullptr ? (a.rows.T + kRowTile - 1) / kRowTile : 0);
    if (grid == 0)
        return cudaSuccess;
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        const auto kernel = a.transposed ? lora_expand_kernel<RP, true> : lora_expand_kernel<RP, false>;
        const int smem = RP * kColTile * 2;
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess)
            return e;
        kernel<<<static_cast<unsigned>(grid), kExpandThreads, smem, stream>>>(a, tiles, col_tiles);
        return cudaGetLastError();
    });
}

cudaError_t launch_lora_outer(const LoraOuterLaunch& a, cudaStream_t stream)
{
    const int in_tiles = (a.hidden_in + kOuterCols - 1) / kOuterCols;
    const int out_tiles = (a.hidden_out + kOuterCols - 1) / kOuterCols;
    return with_rank(a.rank, [&](auto rp) {
        constexpr int RP = decltype(rp)::value;
        const auto kernel = lora_outer_kernel<RP>;
        const int smem = OuterShape<RP>::kBytes;
        const cudaError_t e = allow_smem(kernel, smem);
        if (e != cudaSuccess)
            return e;
        const int64_t grid = static_cast<int64_t>(a.rows.E) * (in_tiles + out_tiles);
        kernel<<<static_cast<unsigned>(grid), kOuterThreads, smem, stream>>>(a, in_tiles, out_tiles);
        return cudaGetLastError();
    });
}

} // namespace ep
