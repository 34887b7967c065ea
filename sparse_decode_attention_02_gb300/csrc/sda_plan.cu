// A step's tables from request lengths: which pages the new tokens take, the
// block table with them, and each new token's slot, position and request.
//
// With c, n the context and new length of request q and B the page size,
//     need = ceil((c + n) / B) - ceil(c / B)
// pages come from the free ring in the order of the requests (an exclusive
// prefix sum of need), token rows likewise (a prefix sum of n).  Every CTA
// computes both sums over all requests (they are small: 8 bytes a request) and
// keeps them in shared memory; the token rows and the page entries are then
// dealt out over the grid and find their request there.  A warp takes 128
// consecutive rows: the requests of the first and the last are searched once for
// all lanes, a lane's own only between those two.  Where there is at most a row a
// thread, each thread finds its own, so that all pages are looked up at once.
//
// A decode step is bound by latency: 256 requests 5.0 us in one CTA, of which about
// 1 us each the lengths, the sums and the grants (the sums are 32-bit and saturate,
// divisions by B are multiplications).  Prompts are bound by the 16 bytes written
// per token row: 4096 of them, 4.2 M rows, 22 us, of which 10 the sums in every CTA
// and 12 the rows, 68 MB at 5.6 TB/s.
#include "sda_common.cuh"

#include <algorithm>

namespace {

using namespace sda;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRequests = 8192;              // six int32 arrays of them in shared memory: 192 KB
constexpr int kArrays = 6;
constexpr size_t kOwnShared = 1024;             // at least the kernel's other shared memory (784 bytes)
constexpr size_t kUsualShared = 48 * 1024;      // what a kernel may use in all before its limit is raised
constexpr int kQuad = 4;                        // consecutive token rows a thread writes at a time
constexpr int kWarpRows = 32 * kQuad;           // rows of a warp's turn
constexpr uint32_t kMostSum = 0x7FFFFFFFu;      // sums stay here: beyond any count of pages or rows
constexpr int kTicketWord = 18;                 // of the workspace header: CTAs past their reads

struct PlanParams {
    const int32_t *context, *added;
    int64_t context_s, added_s;
    int32_t *ring;
    const int32_t *state;
    int32_t *next, *table;
    int64_t table_s0;
    int32_t *seq_lens;
    int64_t seq_s;
    int32_t *starts;
    int64_t *slots;
    int32_t *positions, *owners;
    unsigned int *header;
    int requests, width, block, ring_size, rows;
    int per_request;                            // 0: rows packed; else rows of each request
    unsigned long long inverse;                 // floor(2^64 / block) + 1 (0 for block 1)
    int vec;                                    // the row outputs take 16-byte stores
};

// x / block, exactly, for any 32-bit x.
__device__ __forceinline__ uint32_t pages_before(const PlanParams &p, uint32_t x)
{
    return p.inverse ? static_cast<uint32_t>(__umul64hi(x, p.inverse)) : x;
}

// Three sums over requests: pages needed, pages returned, rows added.
struct Sums {
    uint32_t need, back, add;
};

// A sum that stops at kMostSum; associative for terms up to there.
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b)
{
    return min(a + b, kMostSum);
}

__device__ __forceinline__ Sums operator+(Sums a, Sums b)
{
    return {plus(a.need, b.need), plus(a.back, b.back), plus(a.add, b.add)};
}

__device__ __forceinline__ Sums shfl(Sums v, int lane)
{
    return {__shfl_sync(~0u, v.need, lane), __shfl_sync(~0u, v.back, lane), __shfl_sync(~0u, v.add, lane)};
}

__device__ __forceinline__ Sums warp_inclusive(Sums v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums u = {__shfl_up_sync(~0u, v.need, o), __shfl_up_sync(~0u, v.back, o), __shfl_up_sync(~0u, v.add, o)};
        if (lane >= o)
            v = v + u;
    }
    return v;
}

// The sums over the threads before this one, in thread order, and over all.
__device__ __forceinline__ Sums block_exclusive(const Sums mine, Sums *warp_sums, Sums &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Sums inc = warp_inclusive(mine, lane);
    if (lane == 31)
        warp_sums[warp] = inc;
    __syncthreads();
    const Sums w = warp_inclusive(warp_sums[lane], lane);   // kWarps == 32: a lane a warp
    total = shfl(w, 31);
    const Sums none = {0, 0, 0}, before = shfl(w, max(warp - 1, 0)), left = shfl(inc, max(lane - 1, 0));
    return (warp > 0 ? before : none) + (lane > 0 ? left : none);
}

// The last index in [lo, hi] whose value is at most x (a[lo] <= x; a ascends).
__device__ __forceinline__ int last_at_most(const int32_t *a, int lo, int hi, int x)
{
    int len = hi - lo + 1;
    while (len > 1) {
        const int half = len >> 1;
        lo = a[lo + half] <= x ? lo + half : lo;
        len -= half;
    }
    return lo;
}

// The same for the whole array and one x for the warp: 32 probes at a time.
__device__ __forceinline__ int warp_last_at_most(const int32_t *a, int n, int x, int lane)
{
    int lo = 0;
    while (n > 1) {
        const int stride = (n + 31) >> 5;
        const bool ok = lane * stride < n && a[lo + lane * stride] <= x;
        const int last = __popc(__ballot_sync(~0u, ok)) - 1;
        lo += last * stride;
        n = min(stride, n - last * stride);
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) sda_plan_kernel(const __grid_constant__ PlanParams p)
{
    extern __shared__ int32_t smem[];
    int32_t *ctx = smem;                        // context length
    int32_t *len = ctx + p.requests;            // new length, then the length after the step
    int32_t *tok = len + p.requests;            // token rows before the request
    int32_t *pag = tok + p.requests;            // pages taken before it
    int32_t *rel = pag + p.requests;            // pages returned before it
    int32_t *adj = rel + p.requests;            // pag less the pages the request holds: new column to ring entry
    __shared__ Sums warp_sums[2][kWarps];
    __shared__ int granted[3];                  // token rows, pages taken, pages returned
    __shared__ int is_last;
    static_assert(sizeof warp_sums + sizeof granted + sizeof is_last <= kOwnShared, "shared memory");

    pdl_launch_dependents();
    pdl_wait();

    const int Q = p.requests, B = p.block;
    const int per = (Q + kThreads - 1) / kThreads;
    const int q0 = min(Q, static_cast<int>(threadIdx.x) * per), q1 = min(Q, q0 + per);
    int start = p.state[0], count = p.state[1];
    bool bad = start < 0 || start >= p.ring_size || count < 0 || count > p.ring_size;
    if (bad)
        start = count = 0;
    const bool ring_ok = !bad;
    if (threadIdx.x < 3)
        granted[threadIdx.x] = 0;

    // What request q asks for: pages it needs, pages it returns, rows it adds.
    // Requests outside the contract ask for nothing and raise the flag.
    auto held = [&](int c) { return pages_before(p, static_cast<uint32_t>(max(c, 0)) + (B - 1)); };
    auto asks = [&](int c, int n, Sums &s) {
        s = {0, 0, 0};
        if (n == 0 && c >= 0)
            return true;
        const uint32_t have = held(c);
        if (c < 0 || n < -1 || have > static_cast<uint32_t>(p.width))
            return false;
        if (n == -1) {
            s.back = have;
            return true;
        }
        const uint32_t after = static_cast<uint32_t>(c) + static_cast<uint32_t>(n);
        const uint32_t end = after <= kMostSum ? held(static_cast<int>(after)) : kMostSum;
        if (after > kMostSum || end > static_cast<uint32_t>(p.width) || (p.per_request > 0 && n > p.per_request))
            return false;
        s.need = end - have;
        s.add = n;
        return true;
    };

    Sums mine = {0, 0, 0};
    for (int q = q0; q < q1; ++q) {
        const int c = p.context[q * p.context_s], n = p.added[q * p.added_s];
        Sums s;
        bad = !asks(c, n, s) || bad;
        ctx[q] = c;
        len[q] = n;
        mine = mine + s;
    }
    Sums total;
    Sums run = block_exclusive(mine, warp_sums[0], total);
    if (total.need > static_cast<uint32_t>(count)) {
        // Not all pages are there: rows count only for requests whose pages are.
        uint32_t need = run.need, add = 0;
        for (int q = q0; q < q1; ++q) {
            Sums s;
            asks(ctx[q], len[q], s);
            need = plus(need, s.need);
            add = plus(add, s.need == 0 || need <= static_cast<uint32_t>(count) ? s.add : 0);
        }
        Sums t2;
        run.add = block_exclusive({0, 0, add}, warp_sums[1], t2).add;
    }

    // Grants, in the order of the requests: pages and rows both have to fit.
    // Refusals close a sum's tail, so the granted parts are its beginning.
    bool full = false;
    int top[3] = {0, 0, 0};
    for (int q = q0; q < q1; ++q) {
        const int c = ctx[q], n = len[q];
        Sums s;
        asks(c, n, s);
        tok[q] = static_cast<int>(run.add);
        pag[q] = static_cast<int>(run.need);
        rel[q] = static_cast<int>(run.back);
        adj[q] = static_cast<int>(run.need) - static_cast<int>(held(c));
        run.need = plus(run.need, s.need);
        run.back = plus(run.back, s.back);
        int after = c;
        if (s.add > 0) {
            bool ok = s.need == 0 || run.need <= static_cast<uint32_t>(count);
            run.add = plus(run.add, ok ? s.add : 0);
            ok = ok && run.add <= static_cast<uint32_t>(p.rows);
            if (ok) {
                after = c + n;
                top[0] = static_cast<int>(run.add);
                top[1] = s.need > 0 ? static_cast<int>(run.need) : top[1];
            }
            full = full || !ok;
        } else if (n == -1 && c >= 0 && (s.back > 0 || c == 0)) {
            const bool ok = ring_ok && run.back <= static_cast<uint32_t>(p.ring_size - count);
            if (ok) {
                after = 0;
                top[2] = static_cast<int>(run.back);
            }
            bad = bad || !ok;
        }
        len[q] = after;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int m = __reduce_max_sync(~0u, top[k]);
        if ((threadIdx.x & 31) == 0 && m > 0)
            atomicMax(&granted[k], m);
    }
    const unsigned flags = (bad ? SDA_FLAG_BOUNDS : 0u) | (full ? SDA_FLAG_FULL : 0u);
    const unsigned any = __reduce_or_sync(~0u, flags);
    if ((threadIdx.x & 31) == 0 && any)
        atomicOr(p.header, any);
    __syncthreads();
    const int rows = granted[0], taken = granted[1], returned = granted[2];

    // index into the ring: i < 2 * ring_size
    auto ring_at = [&](uint32_t i) { return i >= static_cast<uint32_t>(p.ring_size) ? i - p.ring_size : i; };

    // The lengths and the ring's state may be updated in place, so they are
    // written by whichever CTA is the last to have read them.
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            const unsigned t = atomicAdd(p.header + kTicketWord, 1u);
            is_last = t == gridDim.x - 1;
            if (is_last)
                p.header[kTicketWord] = 0;
        }
        __syncthreads();
    }
    if (gridDim.x == 1 || is_last) {
        for (int q = threadIdx.x; q < Q; q += kThreads) {
            p.seq_lens[q * p.seq_s] = len[q];
            p.starts[q] = p.per_request > 0 ? (q + 1) * p.per_request - max(len[q] - ctx[q], 0) : min(tok[q], rows);
        }
        if (threadIdx.x == 0) {
            p.starts[Q] = p.per_request > 0 ? p.rows : rows;
            if (ring_ok) {
                p.next[0] = static_cast<int>(ring_at(static_cast<uint32_t>(start + taken)));
                p.next[1] = count - taken + returned;
            } else {
                const int s0 = p.state[0], s1 = p.state[1];
                p.next[0] = s0;
                p.next[1] = s1;
            }
        }
    }

    // ---- Token rows, packed: runs of them, where there is more than one a thread.
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * kWarps, warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int step = gridDim.x * kThreads, me = blockIdx.x * kThreads + threadIdx.x;
    const bool runs = p.per_request == 0 && p.rows > step;
    // a warp's turns are neighbours: its requests follow one another
    const int turns = ((p.rows + kWarpRows - 1) / kWarpRows + warps - 1) / warps;
    int qa = 0, qb = -1;                        // requests of the turn's first and last token row
    for (int turn = 0; turn < turns && runs; ++turn) {
        const long long w = (static_cast<long long>(warp) * turns + turn) * kWarpRows;
        if (w >= p.rows)
            break;
        const int w0 = static_cast<int>(w);
        if (w0 < rows) {
            qa = qb < 0 ? warp_last_at_most(tok, Q, w0, lane) : qb;
            const int last = min(w0 + kWarpRows, rows) - 1;
            int more = 0;
            qb = qa;
            do {                                // tok ascends: the requests that begin by then are a run
                const int q = qb + 1 + lane;
                more = __popc(__ballot_sync(~0u, q < Q && tok[min(q, Q - 1)] <= last));
                qb += more;
            } while (more == 32);
        }
        const int r0 = w0 + lane * kQuad;
        long long slot[kQuad] = {-1, -1, -1, -1};
        int pos[kQuad] = {-1, -1, -1, -1}, own[kQuad] = {-1, -1, -1, -1};
        if (r0 < rows) {
            int q = last_at_most(tok, qa, qb, r0);
            int next = q < qb ? tok[q + 1] : rows;              // row of the next request
            int c = ctx[q], at = c + (r0 - tok[q]);             // the row's position
            int col = static_cast<int>(pages_before(p, static_cast<uint32_t>(at))), off = at - col * B;
            // a column that holds older tokens is the table's, the others come from the ring
            auto page_of = [&] {
                return at - off < c ? p.table[q * p.table_s0 + col]
                                    : p.ring[ring_at(static_cast<uint32_t>(start + adj[q] + col))];
            };
            int page = page_of();
#pragma unroll
            for (int k = 0; k < kQuad; ++k) {
                const int r = r0 + k;
                if (r >= rows)
                    break;
                if (page >= 0)
                    slot[k] = static_cast<long long>(page) * B + off;
                else
                    atomicOr(p.header, SDA_FLAG_BOUNDS);
                pos[k] = at;
                own[k] = q;
                if (k + 1 == kQuad || r + 1 >= rows)
                    break;
                if (r + 1 >= next) {                            // on to the next request with rows
                    do
                        ++q;
                    while (q < qb && tok[q + 1] <= r + 1);
                    next = q < qb ? tok[q + 1] : rows;
                    at = c = ctx[q];
                    col = static_cast<int>(pages_before(p, static_cast<uint32_t>(at)));
                    off = at - col * B;
                    page = page_of();
                } else {
                    ++at;
                    if (++off == B) {
                        off = 0;
                        ++col;
                        page = page_of();
                    }
                }
            }
        }
        if (p.vec && r0 + kQuad <= p.rows) {
            longlong2 *s2 = reinterpret_cast<longlong2 *>(p.slots + r0);
            s2[0] = make_longlong2(slot[0], slot[1]);
            s2[1] = make_longlong2(slot[2], slot[3]);
            *reinterpret_cast<int4 *>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(p.owners + r0) = make_int4(own[0], own[1], own[2], own[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kQuad; ++k)
                if (r0 + k < p.rows) {
                    p.slots[r0 + k] = slot[k];
                    p.positions[r0 + k] = pos[k];
                    p.owners[r0 + k] = own[k];
                }
        }
    }

    // ---- Token rows, each by itself.  So many for each request: its tokens are the
    // last of them.
    for (int r = me; r < p.rows && !runs; r += step) {
        int q, at;                                              // the row's request and position
        bool token;
        if (p.per_request > 0) {
            q = r / p.per_request;
            at = len[q] - ((q + 1) * p.per_request - r);
            token = at >= ctx[q] && len[q] > ctx[q];
        } else {
            token = r < rows;
            q = token ? last_at_most(tok, 0, Q - 1, r) : 0;
            at = token ? ctx[q] + (r - tok[q]) : 0;
        }
        long long slot = -1;
        if (token) {
            const int col = static_cast<int>(pages_before(p, static_cast<uint32_t>(at))), off = at - col * B;
            const int page = at - off < ctx[q] ? p.table[q * p.table_s0 + col]
                                               : p.ring[ring_at(static_cast<uint32_t>(start + adj[q] + col))];
            if (page >= 0)
                slot = static_cast<long long>(page) * B + off;
            else
                atomicOr(p.header, SDA_FLAG_BOUNDS);
        }
        p.slots[r] = slot;
        p.positions[r] = token ? at : -1;
        p.owners[r] = token ? q : -1;
    }

    // In a decode step the first warps write the rows: the last ones begin with the
    // pages taken, those in the middle with the pages returned.
    // ---- Pages taken: their table columns.
    for (int i = step - 1 - me; i < taken; i += step) {
        const int q = last_at_most(pag, 0, Q - 1, i);
        p.table[q * p.table_s0 + (i - adj[q])] = p.ring[ring_at(static_cast<uint32_t>(start + i))];
    }
    // ---- Pages returned: behind the ring's last free page.
    for (int i = me < step / 2 ? me + step / 2 : me - step / 2; i < returned; i += step) {
        const int q = last_at_most(rel, 0, Q - 1, i);
        const uint32_t at = static_cast<uint32_t>(start) + count + i;         // < 2 * ring_size: they fit
        p.ring[ring_at(at)] = p.table[q * p.table_s0 + (i - rel[q])];
    }
}

}  // namespace

extern "C" sda_status sparse_decode_plan_step(const sda_tensor *context_lens, const sda_tensor *new_lens,
                                              int block_size, int rows_per_request,
                                              const sda_tensor *free_pages,
                                              const sda_tensor *free_state, const sda_tensor *free_next,
                                              const sda_tensor *block_table, const sda_tensor *seq_lens,
                                              const sda_tensor *token_starts, const sda_tensor *slots,
                                              const sda_tensor *positions, const sda_tensor *requests,
                                              void *workspace, size_t workspace_bytes, void *stream)
{
    const sda_tensor *vec[] = {context_lens, new_lens, free_pages, free_state, free_next, seq_lens,
                               token_starts, positions, requests};
    for (const sda_tensor *t : vec)
        if (!dims_ok(t, 1) || t->dtype != SDA_DTYPE_INT32)
            return SDA_ERR_INVALID;
    if (!dims_ok(block_table, 2) || block_table->dtype != SDA_DTYPE_INT32 || !dims_ok(slots, 1) ||
        slots->dtype != SDA_DTYPE_INT64)
        return SDA_ERR_INVALID;
    const int64_t Q = context_lens->shape[0], rows = slots->shape[0], ring = free_pages->shape[0];
    if (new_lens->shape[0] != Q || block_table->shape[0] != Q || seq_lens->shape[0] != Q ||
        token_starts->shape[0] != Q + 1 || positions->shape[0] != rows || requests->shape[0] != rows ||
        free_state->shape[0] != 2 || free_next->shape[0] != 2 || ring < 1 || block_size < 1 || rows_per_request < 0 ||
        (rows_per_request > 0 && rows != Q * rows_per_request))
        return SDA_ERR_INVALID;
    const sda_tensor *dense[] = {free_pages, free_state, free_next, token_starts, slots, positions, requests};
    for (const sda_tensor *t : dense)
        if (t->shape[0] > 1 && t->stride[0] != 1)
            return SDA_ERR_INVALID;
    if (block_table->shape[1] > 1 && block_table->stride[1] != 1)
        return SDA_ERR_INVALID;
    // Written tensors must not be broadcast over requests.
    if (Q > 1 && (seq_lens->stride[0] == 0 || block_table->stride[0] < block_table->shape[1]))
        return SDA_ERR_INVALID;
    if (Q > kMaxRequests || ring > (1 << 30) || rows > (1 << 30) || block_table->shape[1] > INT32_MAX)
        return SDA_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < kHeaderBytes)
        return SDA_ERR_WORKSPACE;
    for (const sda_tensor *t : dense)
        if (t->shape[0] > 0 && !t->data)
            return SDA_ERR_INVALID;
    if (Q > 0 && (!context_lens->data || !new_lens->data || !seq_lens->data ||
                  (block_table->shape[1] > 0 && !block_table->data)))
        return SDA_ERR_INVALID;

    PlanParams p = {};
    p.context = static_cast<const int32_t *>(context_lens->data);
    p.context_s = context_lens->stride[0];
    p.added = static_cast<const int32_t *>(new_lens->data);
    p.added_s = new_lens->stride[0];
    auto out32 = [](const sda_tensor *t) { return static_cast<int32_t *>(const_cast<void *>(t->data)); };
    p.ring = out32(free_pages);
    p.state = static_cast<const int32_t *>(free_state->data);
    p.next = out32(free_next);
    p.table = out32(block_table);
    p.table_s0 = block_table->stride[0];
    p.seq_lens = out32(seq_lens);
    p.seq_s = seq_lens->stride[0];
    p.starts = out32(token_starts);
    p.slots = static_cast<int64_t *>(const_cast<void *>(slots->data));
    p.positions = out32(positions);
    p.owners = out32(requests);
    p.header = static_cast<unsigned int *>(workspace);
    p.requests = static_cast<int>(Q);
    p.width = static_cast<int>(block_table->shape[1]);
    p.block = block_size;
    p.ring_size = static_cast<int>(ring);
    p.rows = static_cast<int>(rows);
    p.per_request = rows_per_request;
    p.inverse = block_size > 1 ? ~0ull / static_cast<unsigned>(block_size) + 1 : 0;
    p.vec = aligned(p.slots, 16) && aligned(p.positions, 16) && aligned(p.owners, 16);

    const size_t smem = kArrays * sizeof(int32_t) * static_cast<size_t>(Q);
    static size_t raised[64] = {};
    if (smem + kOwnShared > kUsualShared && !raise_smem(sda_plan_kernel, kArrays * sizeof(int32_t) * kMaxRequests, raised))
        return SDA_ERR_CUDA;
    const int sms = sm_count();
    if (sms < 1)
        return SDA_ERR_CUDA;
    // One CTA while its warps have one turn of rows each (460,000 rows of 1021 requests:
    // 113 CTAs, 9.0 us); else a turn per warp, up to a CTA an SM.
    const int64_t want = (rows + kWarps * kWarpRows - 1) / (kWarps * kWarpRows);
    const int grid = static_cast<int>(std::min<int64_t>(sms, std::max<int64_t>(1, want)));
    return launch_pdl(sda_plan_kernel, dim3(grid), dim3(kThreads), smem, stream, p);
}
