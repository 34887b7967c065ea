// Host side of the paged attention, and the kernel that joins the pieces of a
// request that several CTAs computed.
#include "sda_context.cuh"
#include "sda_paged.cuh"

#include <cmath>
#include <cstring>
#include <mutex>
#include <numeric>

namespace {

using namespace sda;
using namespace sda::paged;

// ---------------------------------------------------------------------------
// Join kernel.  With partial outputs O_k and their log-sum-exps L_k,
//     o = sum_k e^(L_k - M) O_k / sum_k e^(L_k - M),  L = M + log of that sum.
// The split kernel lists what is to be joined, so the work does not grow with
// the batch.  A row of few pieces is one warp's; one of many (a request alone on
// the GPU leaves a piece per worker) is shared by a block's warps, which add up
// through shared memory in a fixed order.  It reads each partial once (some MB, in
// L2) and is bound by latency: about 6 us of the 76 of one long request, 2 of them
// the launch.
// ---------------------------------------------------------------------------

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <int D, int UNROLL>                    // pieces loaded at a time
__global__ void __launch_bounds__(kJoinThreads) sda_paged_join_kernel(const __grid_constant__ Params p)
{
    constexpr int kVecs = D / 64;               // pairs of dims a lane has
    __shared__ float2 sums[kJoinWarps][D / 2];
    __shared__ int list_piece[kMaxWorkers], counts[kJoinWarps];
    __shared__ float list_lse[kMaxWorkers];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = min(static_cast<int>(p.flags[kItemWord]), kMaxItems), H = p.heads;
    JoinItem next = p.items[min(static_cast<int>(blockIdx.x), kMaxItems - 1)];     // beside the count: one latency
    for (int i = blockIdx.x; i < count; i += gridDim.x) {
        const JoinItem item = next;
        if (i + static_cast<int>(gridDim.x) < count)
            next = p.items[i + gridDim.x];
        const int n = item.pieces;
        // what no split kernel wrote (a workspace whose header was not zeroed) is left out
        if (n < 1 || item.rows < 1 || item.first < 0 || item.first > p.workers - n || item.request < 0 || item.request >= p.requests ||
            item.group < 0 || item.group >= p.groups || item.row < 0 || item.row > p.rows - item.rows)
            continue;
        const bool shared = n > kManyPieces;
        const int r = item.row + (shared ? 0 : warp);
        if (!shared && warp >= item.rows)
            continue;
        // piece k: the first worker's part goes on, the others' continue it
        auto place = [&](int k) {
            return ((static_cast<int64_t>(item.first) + k) * 2 + (k == 0 ? 1 : 0)) * p.rows + r;
        };
        const int j = (r * p.head_inv) >> 16, h = r - j * H;
        const int64_t token = static_cast<int64_t>(item.request) * p.query_len + j;
        // regions: an item's request is a row
        const int64_t gate_token = p.region_groups ? item.request / p.region_groups : token;
        const int gate_group = p.region_groups ? item.request % p.region_groups : item.group;
        const uint16_t *gate =
            p.gate ? p.gate + gate_token * p.g_s0 + static_cast<int64_t>(gate_group * H + h) * p.g_s1 : nullptr;
        const uint16_t gate_bits = gate ? *gate : 0;            // beside what follows
        const float vs = p.v_scale ? *p.v_scale : 1.0f;

        // The pieces that saw a token (and were not merged into a neighbour's),
        // in order: bits and a lane each, or a list in shared memory.
        unsigned have = 0;
        int live = 0;
        float l = -INFINITY;
        if (!shared) {
            l = lane < n ? p.part_lse[place(lane)] : -INFINITY;
            have = __ballot_sync(~0u, l != -INFINITY);
        } else {
            auto lse_of = [&](int k) { return k < n ? p.part_lse[place(k)] : -INFINITY; };
            const int k1 = static_cast<int>(threadIdx.x);
            float next_x = lse_of(k1 + kJoinThreads), x = lse_of(k1);     // a turn ahead
            for (int k0 = 0; k0 < n; k0 += kJoinThreads, x = next_x, next_x = lse_of(k1 + k0 + kJoinThreads)) {
                const int k = k0 + k1;
                const unsigned some = __ballot_sync(~0u, x != -INFINITY);
                __syncthreads();                // the list and counts of the last round, or item, have been read
                if (lane == 0)
                    counts[warp] = __popc(some);
                __syncthreads();
                int at = live + __popc(some & ((1u << lane) - 1u));
                for (int w = 0; w < kJoinWarps; ++w) {
                    at += w < warp ? counts[w] : 0;
                    live += counts[w];
                }
                if (x != -INFINITY) {
                    list_piece[at] = k;
                    list_lse[at] = x;
                }
            }
            __syncthreads();
        }
        float M = l;
        for (int k = lane; k < live; k += 32)
            M = fmaxf(M, list_lse[k]);
        M = warp_max(M);
        const float ref = M == -INFINITY ? 0.0f : M;
        float W = shared ? 0.0f : exp2f(l - ref);
        for (int k = lane; k < live; k += 32)
            W += exp2f(list_lse[k] - ref);
        W = warp_sum(W);

        float2 acc[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            acc[i] = make_float2(0.0f, 0.0f);
        int at = warp;                          // of the list
        while (have != 0 || at < live) {
            float2 x[UNROLL][kVecs];
            float w[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const bool some = shared ? at < live : have != 0;
                const int k = !some ? 0 : shared ? list_piece[at] : __ffs(have) - 1;
                w[u] = shared ? (some ? list_lse[at] : 0.0f) : __shfl_sync(~0u, l, k);
                w[u] = some ? w[u] : -INFINITY;
                const float2 *src = reinterpret_cast<const float2 *>(p.partial + place(k) * D) + lane;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    x[u][i] = some ? src[32 * i] : make_float2(0.0f, 0.0f);
                have &= have - 1;
                at += kJoinWarps;
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const float f = exp2f(w[u] - ref);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    acc[i].x += f * x[u][i].x;
                    acc[i].y += f * x[u][i].y;
                }
            }
            if (!shared)
                at = 0;
        }
        if (shared) {
            // the last item's sums were read before this item's list was made
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                sums[warp][32 * i + lane] = acc[i];
            __syncthreads();
            if (warp > 0)
                continue;
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    acc[i].x += sums[w][32 * i + lane].x;
                    acc[i].y += sums[w][32 * i + lane].y;
                }
        }

        const bool empty = M == -INFINITY && W == 0.0f;         // a row that saw no token; NaN goes on
        const int64_t row = token * p.groups + item.group;
        const float f = empty ? 0.0f : vs / W * (gate ? gate_factor(gate_bits) : 1.0f);
        uint16_t *dst = p.output + row * p.o_s0 + h * p.o_s1 + 2 * lane;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t w = pack_bf16(acc[i].x * f, acc[i].y * f);
            if (p.o_vec) {
                *reinterpret_cast<uint32_t *>(dst + 64 * i) = w;
            } else {
                dst[64 * i] = static_cast<uint16_t>(w);
                dst[64 * i + 1] = static_cast<uint16_t>(w >> 16);
            }
        }
        if (p.lse && lane == 0)
            p.lse[row * p.l_s0 + h * p.l_s1] = empty ? -INFINITY : (M + log2f(W)) * kLn2;
    }
    // The list is empty again for the next call once every block has read its length.
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.flags + kTicketWord, 1u) == gridDim.x - 1) {
        p.flags[kItemWord] = 0;
        p.flags[kTicketWord] = 0;
    }
}

// ---------------------------------------------------------------------------
// Extent kernel: how far a row's list of regions has one that the row sees.  Lists end in
// -1 where a context has fewer regions than are selected; dealt out by their room alone
// such rows would leave most workers idle.  A warp a row, from the end on: of a full list
// the last ids are all that it reads.  2 to 3 us, most of it the launch.
// ---------------------------------------------------------------------------

constexpr int kExtentWarps = 4, kExtentIds = 4;                 // ids of a lane at a time

__global__ void __launch_bounds__(kExtentWarps * 32) sda_region_extent_kernel(const __grid_constant__ Params p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kExtentWarps + (threadIdx.x >> 5);
    if (row >= p.requests)
        return;
    const int32_t *ids = p.regions + row * p.reg_s0;
    int id[kExtentIds];                         // the list's last ones, beside the row's position and flag: one latency
    auto load = [&](int end) {
#pragma unroll
        for (int k = 0; k < kExtentIds; ++k) {
            const int i = end - 1 - 32 * k - lane;
            id[k] = i >= 0 ? ids[i] : -1;
        }
    };
    load(p.listed);
    const int pos = p.positions[row * p.pos_s];
    const bool active = p.active[row * p.act_s] != 0;
    int last = -1;
    if (active) {
        const int most = pos >= 0 ? pos / p.region_tokens : -1;               // the last region that it sees
        for (int end = p.listed; end > 0 && last < 0; end -= 32 * kExtentIds) {
            if (end < p.listed)
                load(end);
#pragma unroll
            for (int k = 0; k < kExtentIds; ++k) {
                if (id[k] < -1)
                    atomicOr(p.flags, SDA_FLAG_BOUNDS);
                const unsigned live = __ballot_sync(~0u, id[k] >= 0 && id[k] <= most);
                if (last < 0 && live)
                    last = end - 1 - 32 * k - (__ffs(live) - 1);
            }
        }
    }
    if (lane == 0)
        p.extents[row] = active ? (last + 1) * p.region_tokens : p.clear_inactive ? 0 : -1;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

bool dim_ok(int64_t d)
{
    return d == 64 || d == 128 || d == 192 || d == 256;
}

size_t align256(size_t n)
{
    return (n + 255) & ~static_cast<size_t>(255);
}

// Units of at most kWholeTiles tiles (by the table's width) are never cut: a worker
// takes them whole.  A CTA takes a unit alone instead
//   * up to kAloneTiles tiles a worker (2 groups; cut and joined against alone: bf16,
//     192 dims, 63 tiles, 1 request 14.6, 17.6 us, 76 requests 31.9, 24.3; 80 E4M3
//     requests of 100 to 2300 tokens, 72 tiles, 27.5, 35.5: lengths that differ lose
//     what equal ones gain), or twice that with more than 16 query rows, whose
//     pieces are large, and units for every CTA (E4M3, 192 dims, 64 rows: 400
//     requests of up to 700 tokens 113.6, 88.9; 80 of 100 to 700 33.6, 41.0);
//   * in at most kRounds rounds of CTAs (1500 E4M3 requests of up to 900 tokens x 2
//     groups: 105 us cut, 126 alone), or one where a worker could take it whole (600
//     bf16 requests of 96 tokens, 192 dims: 21 us whole, 29 alone; 8 of 16 tokens,
//     in one round: 7.4, 5.8).
constexpr int kWholeTiles = 8, kAloneTiles = 12;
constexpr int kRounds = 4;
// Few units of a quantised cache are taken by clusters: more than kFewTiles tiles for each of
// one CTA's workers and at most kClusterTiles for each of the cluster's (E4M3, 192 dims, 4 groups;
// without, with: one request of 600 tokens 12.1 us, 10.9, of 1200 17.1, 11.6, of 5000 16.7, 15.2;
// with two new tokens 700 20.0, 11.3; 16 requests of 300 to 1200 17.9, 15.6; six rows of 32 regions
// of 64 in integers 16.2, 12.9.  With fewer tiles, one of 300 9.6, 11.1; with more, one of 10,000 18.7, 20.8).
constexpr int kFewTiles = 4, kClusterTiles = 8;
// Rows' lists are looked at for their extents where a worker has at least this many tiles of their
// room (1024 slots, E4M3, 192 dims, 2 groups; not looked at, looked at: 256 requests of 1K to 2K tokens
// 192 us, 90, of 16K to 32K 284, 292; 16 requests of 1K to 3K 32.4, 26.6, of 16K to 20K 38.4, 40.0;
// four of either, which have fewer tiles, 19.3 and 20.6, and 24.1 and 22.6).
constexpr int kExtentTiles = 8;

// CTAs of a launch, at most.
int ctas_of(int64_t dim, int64_t rows)
{
    return kSms * ctas_per_sm(static_cast<int>(dim), tiles_of_rows(static_cast<int>(rows)));
}

// Workers of a CTA.
int workers_of(int64_t rows)
{
    return kWarps / tiles_of_rows(static_cast<int>(rows));
}

}  // namespace

extern "C" size_t sparse_decode_quantised_workspace_bytes(int64_t rows, int heads, int head_dim)
{
    const size_t bytes = heads <= kMaxRegionHeads ? sparse_decode_paged_workspace_bytes(heads, 1, head_dim) : 0;
    return bytes && rows >= 0 && rows <= INT32_MAX ? bytes + align256(static_cast<size_t>(rows) * sizeof(int32_t)) : 0;
}

extern "C" size_t sparse_decode_paged_workspace_bytes(int heads, int query_len, int head_dim)
{
    if (heads < 1 || query_len < 1 || heads > kMaxRows || query_len > kMaxRows || heads * query_len > kMaxRows ||
        !dim_ok(head_dim))
        return 0;
    const size_t rows = static_cast<size_t>(ctas_of(head_dim, heads * query_len)) * workers_of(heads * query_len) * 2 *
                        heads * query_len;
    return kHeaderBytes + align256(kItemBytes) + rows * head_dim * sizeof(float) + align256(rows * sizeof(float));
}

namespace {

// One call of the entry points below after argument unpacking: whole caches
// (seq_lens) or regions (regions, positions, active), plain caches (k_scale and
// v_scale beside E4M3) or quantised ones (scales).
struct Call {
    const sda_tensor *query, *cache, *scales, *block_table, *seq_lens, *output, *lse, *gate;
    const sda_tensor *regions, *positions, *active;
    float scale;
    int query_len, clear_inactive, region_tokens;
    const float *k_scale, *v_scale;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
};

sda_status run_call(const Call &c)
{
    const sda_tensor *query = c.query, *cache = c.cache, *block_table = c.block_table, *output = c.output;
    const bool by_region = c.regions != nullptr;
    // ---- Contract.
    if (!dims_ok(query, 3) || !dims_ok(cache, 4) || !dims_ok(block_table, 2) || !dims_ok(output, 3) ||
        (by_region ? !dims_ok(c.regions, 2) || !dims_ok(c.positions, 1) || !dims_ok(c.active, 1) : !dims_ok(c.seq_lens, 1)))
        return SDA_ERR_INVALID;
    const int64_t rows = query->shape[0], heads = query->shape[1], dim = query->shape[2];
    if (query->dtype != SDA_DTYPE_BF16 || output->dtype != SDA_DTYPE_BF16 || block_table->dtype != SDA_DTYPE_INT32)
        return SDA_ERR_INVALID;
    if (by_region ? c.regions->dtype != SDA_DTYPE_INT32 || c.positions->dtype != SDA_DTYPE_INT32 ||
                        (c.active->dtype != SDA_DTYPE_BOOL && c.active->dtype != SDA_DTYPE_UINT8)
                  : c.seq_lens->dtype != SDA_DTYPE_INT32)
        return SDA_ERR_INVALID;
    const bool fp8 = !c.scales && is_fp8(cache);
    if (!c.scales && !fp8 && cache->dtype != SDA_DTYPE_BF16)
        return SDA_ERR_INVALID;
    if (cache->shape[3] != 2 * dim || output->shape[0] != rows || output->shape[1] != heads ||
        output->shape[2] != dim)
        return SDA_ERR_INVALID;
    if (query->stride[2] != 1 || output->stride[2] != 1 || cache->stride[3] != 1 ||
        (block_table->shape[1] > 1 && block_table->stride[1] != 1))
        return SDA_ERR_INVALID;
    if (!dim_ok(dim) || heads < 1 || heads > (by_region ? kMaxRegionHeads : kMaxRows))
        return SDA_ERR_UNSUPPORTED;
    if (c.query_len < 1 || !std::isfinite(c.scale) || (fp8 && (!c.k_scale || !c.v_scale)))
        return SDA_ERR_INVALID;
    // Query rows of a unit: a request's tokens, or one row of regions.
    const int query_len = by_region ? 1 : c.query_len;
    if (heads * query_len > kMaxRows)
        return SDA_ERR_UNSUPPORTED;
    QuantisedCache quantised = {};
    if (c.scales) {
        const sda_status st = check_quantised(cache, c.scales, dim, quantised);
        if (st != SDA_OK)
            return st;
    }
    const int64_t pages = cache->shape[0], groups = cache->shape[1], block = cache->shape[2];
    if (groups < 1 || block < 1 || pages < 1)
        return SDA_ERR_INVALID;
    int64_t requests, units;                    // lines of the table; units that the kernel is to cut
    if (by_region) {
        requests = (rows + groups * c.query_len - 1) / (groups * c.query_len);
        units = rows;
        if (rows % groups != 0 || block_table->shape[0] < requests || c.regions->shape[0] != rows ||
            c.positions->shape[0] != rows || c.active->shape[0] != rows ||
            (c.regions->shape[1] > 1 && c.regions->stride[1] != 1) || c.region_tokens < 0)
            return SDA_ERR_INVALID;
    } else {
        requests = c.seq_lens->shape[0];
        units = requests * groups;
        if (rows % (groups * query_len) != 0 || rows / (groups * query_len) != requests || block_table->shape[0] < requests)
            return SDA_ERR_INVALID;
    }
    const bool gated = given(c.gate);
    if (gated && (!dims_ok(c.gate, 2) || c.gate->dtype != SDA_DTYPE_BF16 || c.gate->shape[0] != rows / groups ||
                  c.gate->shape[1] != groups * heads))
        return SDA_ERR_INVALID;
    const bool with_lse = given(c.lse);
    if (with_lse && (!dims_ok(c.lse, 2) || c.lse->dtype != SDA_DTYPE_FP32 || c.lse->shape[0] != rows ||
                     c.lse->shape[1] != heads || (rows > 1 && c.lse->stride[0] == 0) ||
                     (heads > 1 && c.lse->stride[1] == 0)))
        return SDA_ERR_INVALID;
    if ((rows > 1 && output->stride[0] == 0) || (heads > 1 && output->stride[1] == 0))
        return SDA_ERR_INVALID;
    if (pages > INT32_MAX || rows > INT32_MAX / kMaxRows || block_table->shape[1] > INT32_MAX ||
        block > (1 << 24) || groups > (1 << 16))
        return SDA_ERR_UNSUPPORTED;
    const int elt = cache->dtype == SDA_DTYPE_BF16 ? 2 : 1, row_bytes = static_cast<int>(2 * dim) * elt;
    if (block % 8 != 0)
        return SDA_ERR_UNSUPPORTED;
    if (!aligned(cache->data, 16))
        return SDA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (cache->stride[i] <= 0 || (cache->stride[i] * elt) % 16 != 0)
            return SDA_ERR_UNSUPPORTED;
    // Pieces divide pages, and regions.
    const int64_t region = by_region ? (c.region_tokens ? c.region_tokens : block) : 0;
    const int64_t whole = by_region ? std::gcd(region, block) : block;
    if (by_region && (whole % 8 != 0 || region > (1 << 24) || c.regions->shape[1] > (1 << 20) ||
                      c.regions->shape[1] * region > INT32_MAX - 4096))
        return SDA_ERR_UNSUPPORTED;
    const int64_t held = by_region ? c.regions->shape[1] * region : block_table->shape[1] * block;
    const size_t need = by_region ? sparse_decode_quantised_workspace_bytes(rows, static_cast<int>(heads), static_cast<int>(dim))
                                  : sparse_decode_paged_workspace_bytes(static_cast<int>(heads), query_len, static_cast<int>(dim));
    if (!c.workspace || !aligned(c.workspace, 256) || c.workspace_bytes < need)
        return SDA_ERR_WORKSPACE;
    if (rows == 0)
        return SDA_OK;
    if (!query->data || !cache->data || !output->data || (!block_table->data && block_table->shape[1] > 0) ||
        (c.scales && !c.scales->data))
        return SDA_ERR_INVALID;
    if (by_region ? !c.positions->data || !c.active->data || (!c.regions->data && c.regions->shape[1] > 0)
                  : !c.seq_lens->data)
        return SDA_ERR_INVALID;

    // ---- How the work is split, by the tiles that a request can have at most.
    const int sms = sm_count();
    if (sms < 1)
        return SDA_ERR_CUDA;
    Params p = {};
    p.rows = static_cast<int>(heads) * query_len;
    p.cap = static_cast<int>(std::min<int64_t>(held, INT32_MAX - 4096));
    const int mt = tiles_of_rows(p.rows), per_cta = workers_of(p.rows);
    const int most = std::min(ctas_of(dim, p.rows), ctas_per_sm(static_cast<int>(dim), mt) * sms);
    // A TMA box holds the longest run of tokens that fits a stage and divides the
    // page, a tile the boxes that fit.  The tiles of the table's width:
    auto widest_with = [&](bool alone) {
        const int slots = stage_slots(row_bytes, mt, alone);
        p.piece = static_cast<int>(std::min<int64_t>(whole, slots)) / 8 * 8;
        while (whole % p.piece != 0)
            p.piece -= 8;
        p.tile = slots / p.piece * p.piece;
        return (p.cap + static_cast<int64_t>(p.tile) - 1) / p.tile;
    };
    int64_t widest = widest_with(true);
    // A cluster is as large as leaves an SM to each CTA and a tile to each worker.
    p.cluster = 1;
    if (c.scales && mt <= 2 && widest > kFewTiles * per_cta)
        while (p.cluster < kMaxCluster && units * p.cluster * 2 <= sms && p.cluster * 2 * per_cta <= widest)
            p.cluster *= 2;
    if (p.cluster > 1 && widest > kClusterTiles * p.cluster * per_cta)
        p.cluster = 1;
    p.cta_units = p.cluster > 1 ||
                  (widest <= (per_cta < kWarps && units >= most ? 2 : 1) * kAloneTiles * per_cta &&
                   units <= (widest > kWholeTiles ? kRounds : 1) * static_cast<int64_t>(most));
    if (!p.cta_units)
        widest = widest_with(false);
    p.whole_units = !p.cta_units && widest <= kWholeTiles;
    // Few tiles: a worker on each of as many SMs first.
    const int cost = unit_cost(c.scales != nullptr);
    const int64_t want = p.whole_units || p.cta_units ? units : (units * (widest + cost) - 1) / (kMinTiles + cost) + 1;
    p.ctas = static_cast<int>(p.cta_units ? units * p.cluster : std::min<int64_t>(most, std::max<int64_t>(1, want)));
    p.workers = p.ctas * per_cta;

    // ---- The cache as (128 bytes, token, band, group, page): a box is a piece
    // of all bands, landing as [band][token][128 bytes], swizzled.
    EncodeTiledFn encode = encode_fn();
    if (!encode)
        return SDA_ERR_CUDA;
    CUtensorMap tmap;
    const int bands = row_bytes / 128;
    const cuuint64_t gdim[5] = {static_cast<cuuint64_t>(128 / elt), static_cast<cuuint64_t>(block),
                                static_cast<cuuint64_t>(bands), static_cast<cuuint64_t>(groups),
                                static_cast<cuuint64_t>(pages)};
    const cuuint64_t gstride[4] = {static_cast<cuuint64_t>(cache->stride[2] * elt), 128u,
                                   static_cast<cuuint64_t>(cache->stride[1] * elt),
                                   static_cast<cuuint64_t>(cache->stride[0] * elt)};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(128 / elt), static_cast<cuuint32_t>(p.piece),
                               static_cast<cuuint32_t>(bands), 1, 1};
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    if (with_context(encode, &tmap, elt == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                     const_cast<void *>(cache->data), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return SDA_ERR_UNSUPPORTED;

    p.query = static_cast<const uint16_t *>(query->data);
    p.q_s0 = query->stride[0];
    p.q_s1 = query->stride[1];
    p.block_table = static_cast<const int32_t *>(block_table->data);
    p.bt_s0 = block_table->stride[0];
    if (by_region) {
        p.regions = static_cast<const int32_t *>(c.regions->data);
        p.reg_s0 = c.regions->stride[0];
        p.positions = static_cast<const int32_t *>(c.positions->data);
        p.pos_s = c.positions->stride[0];
        p.active = static_cast<const uint8_t *>(c.active->data);
        p.act_s = c.active->stride[0];
        p.region_tokens = static_cast<int>(region);
        p.listed = static_cast<int>(c.regions->shape[1]);
        p.block_inv = inverse_of(static_cast<unsigned>(block));
        p.per_region = static_cast<int>(region / p.piece);
        p.per_region_inv = inverse_of(static_cast<unsigned>(p.per_region));
        p.region_groups = static_cast<int>(groups);
        p.region_groups_inv = inverse_of(static_cast<unsigned>(groups));
        // a line of the table for all rows where a request has as many as there are
        p.request_rows = static_cast<int>(std::min<int64_t>(groups * c.query_len, INT32_MAX));
        p.request_rows_inv = inverse_of(static_cast<unsigned>(p.request_rows));
        p.clear_inactive = c.clear_inactive ? 1 : 0;
    } else {
        p.seq_lens = static_cast<const int32_t *>(c.seq_lens->data);
        p.len_s = c.seq_lens->stride[0];
    }
    if (c.scales) {
        p.scales = static_cast<const float *>(c.scales->data);
        p.s_s0 = c.scales->stride[0], p.s_s1 = c.scales->stride[1], p.s_s2 = c.scales->stride[2];
        p.span_inv = inverse_of(static_cast<unsigned>(quantised.span));
        p.one_scale = quantised.span % p.piece == 0;
    }
    p.output = static_cast<uint16_t *>(const_cast<void *>(output->data));
    p.o_s0 = output->stride[0];
    p.o_s1 = output->stride[1];
    if (with_lse) {
        p.lse = static_cast<float *>(const_cast<void *>(c.lse->data));
        p.l_s0 = c.lse->stride[0];
        p.l_s1 = c.lse->stride[1];
    }
    if (gated) {
        p.gate = static_cast<const uint16_t *>(c.gate->data);
        p.g_s0 = c.gate->stride[0];
        p.g_s1 = c.gate->stride[1];
    }
    p.k_scale = fp8 ? c.k_scale : nullptr;
    p.v_scale = fp8 ? c.v_scale : nullptr;
    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    const size_t parts = static_cast<size_t>(ctas_of(dim, heads * query_len)) * per_cta * 2 * heads * query_len;
    p.flags = reinterpret_cast<unsigned int *>(ws);
    p.items = reinterpret_cast<JoinItem *>(ws + kHeaderBytes);
    p.partial = reinterpret_cast<float *>(ws + kHeaderBytes + align256(kItemBytes));
    p.part_lse = p.partial + parts * dim;
    p.pages = pages;
    p.wait_ns = sda_wait_limit_ns();
    p.scale = c.scale;
    p.requests = static_cast<int>(by_region ? rows : requests);
    p.groups = static_cast<int>(by_region ? 1 : groups);
    p.heads = static_cast<int>(heads);
    p.head_inv = (65536 + p.heads - 1) / p.heads;
    p.query_len = query_len;
    p.table_cols = static_cast<int>(block_table->shape[1]);
    p.block = static_cast<int>(block);
    auto runs_of_4 = [](const sda_tensor *t) {
        return aligned(t->data, 8) && t->stride[0] % 4 == 0 && t->stride[1] % 4 == 0;
    };
    p.q_vec = runs_of_4(query);
    p.o_vec = runs_of_4(output);

    p.workers_inv = inverse_of(static_cast<unsigned>(p.workers));
    p.tile_inv = inverse_of(static_cast<unsigned>(p.tile));
    p.per_block_inv = inverse_of(static_cast<unsigned>(p.block / p.piece));

    static Launch *const kLaunches[6][4] = {
        {launch_bf16_64, launch_bf16_128, launch_bf16_192, launch_bf16_256},
        {launch_fp8_64, launch_fp8_128, launch_fp8_192, launch_fp8_256},
        {launch_qe4m3_64, launch_qe4m3_128, launch_qe4m3_192, launch_qe4m3_256},
        {launch_qint8_64, launch_qint8_128, launch_qint8_192, launch_qint8_256},
        {regions_qe4m3_64, regions_qe4m3_128, regions_qe4m3_192, regions_qe4m3_256},
        {regions_qint8_64, regions_qint8_128, regions_qint8_192, regions_qint8_256}};
    const int kind = c.scales ? 2 + (quantised.int8 ? 1 : 0) + (by_region ? 2 : 0) : fp8 ? 1 : 0;
    Launch *launch = kLaunches[kind][dim / 64 - 1];
    // The split kernel leaves its list and pieces in the workspace, the join empties it.
    const std::lock_guard<std::mutex> together(sda_launch_mutex(c.workspace));
    if (by_region && !p.whole_units && !p.cta_units && units * widest >= kExtentTiles * static_cast<int64_t>(p.workers)) {
        p.extents = reinterpret_cast<int32_t *>(
            ws + sparse_decode_paged_workspace_bytes(static_cast<int>(heads), query_len, static_cast<int>(dim)));
        const dim3 blocks(static_cast<unsigned>((rows + kExtentWarps - 1) / kExtentWarps));
        const sda_status looked = launch_pdl(sda_region_extent_kernel, blocks, dim3(kExtentWarps * 32), 0, c.stream, p);
        if (looked != SDA_OK)
            return looked;
    }
    const sda_status st = launch(tmap, p, c.stream);
    if (st != SDA_OK || p.whole_units || p.cta_units)
        return st;
    // A block an item (at most eight rows of a unit) as long as they run together.
    const int64_t items = units * ((p.rows + kJoinWarps - 1) / kJoinWarps);
    const int64_t rows_to_join = units <= p.workers / kManyPieces ? units * p.rows : items;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(4 * sms, rows_to_join)));
    // Eight pieces at a time where each SM has a row at most (one request of 261,001
    // tokens: 78.7 us with four, 77.4 with eight), four where registers decide how
    // many rows there are at a time (188 requests of up to 2500: 56.3, 59.9; 256 dims,
    // 96 rows: 51.1, 52.3).
    const bool few = units * p.rows <= sms;
    auto join = dim == 64    ? (few ? sda_paged_join_kernel<64, 8> : sda_paged_join_kernel<64, 4>)
                : dim == 128 ? (few ? sda_paged_join_kernel<128, 8> : sda_paged_join_kernel<128, 4>)
                : dim == 192 ? (few ? sda_paged_join_kernel<192, 8> : sda_paged_join_kernel<192, 4>)
                             : sda_paged_join_kernel<256, 4>;
    return launch_pdl(join, grid, dim3(kJoinThreads), 0, c.stream, p);
}

}  // namespace

extern "C" sda_status sparse_decode_paged_attention(const sda_tensor *query, const sda_tensor *cache,
                                                    const sda_tensor *block_table, const sda_tensor *seq_lens,
                                                    const sda_tensor *output, const sda_tensor *lse, float scale,
                                                    int query_len, const float *k_scale, const float *v_scale,
                                                    const sda_tensor *gate, void *workspace,
                                                    size_t workspace_bytes, void *stream)
{
    return run_call({query, cache, nullptr, block_table, seq_lens, output, lse, gate, nullptr, nullptr, nullptr, scale,
                     query_len, 0, 0, k_scale, v_scale, workspace, workspace_bytes, stream});
}

extern "C" sda_status sparse_decode_quantised_paged_attention(const sda_tensor *query, const sda_tensor *cache,
                                                              const sda_tensor *scales, const sda_tensor *block_table,
                                                              const sda_tensor *seq_lens, const sda_tensor *output,
                                                              const sda_tensor *lse, float scale, int query_len,
                                                              const sda_tensor *gate, void *workspace,
                                                              size_t workspace_bytes, void *stream)
{
    if (!scales)
        return SDA_ERR_INVALID;
    return run_call({query, cache, scales, block_table, seq_lens, output, lse, gate, nullptr, nullptr, nullptr, scale,
                     query_len, 0, 0, nullptr, nullptr, workspace, workspace_bytes, stream});
}

extern "C" sda_status sparse_decode_quantised_attention(const sda_tensor *query, const sda_tensor *cache,
                                                        const sda_tensor *scales, const sda_tensor *regions,
                                                        const sda_tensor *block_table, const sda_tensor *positions,
                                                        const sda_tensor *active, const sda_tensor *output,
                                                        const sda_tensor *lse, float scale, int query_len,
                                                        const sda_tensor *gate, int clear_inactive, int region_tokens,
                                                        void *workspace, size_t workspace_bytes, void *stream)
{
    if (!scales || !regions || !positions || !active)
        return SDA_ERR_INVALID;
    return run_call({query, cache, scales, block_table, nullptr, output, lse, gate, regions, positions, active, scale,
                     query_len, clear_inactive, region_tokens, nullptr, nullptr, workspace, workspace_bytes, stream});
}
