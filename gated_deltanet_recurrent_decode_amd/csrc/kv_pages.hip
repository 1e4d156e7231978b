// kv_pages.hip -- the pages of a KV cache on the device (gfx950): growing,
// forking and ending rows, copying and packing pages.
//
// The cache's counterpart of slot_ops.hip and slot_commit.hip: bookkeeping in
// stream order, nothing read back to the host.  What hands out pages runs in one
// workgroup, so the order of the list, and with it every table, is the same each
// time: needs are summed over the list, the free pages' numbers are listed in
// ascending order until they suffice, and entry i takes those from its sum on.
// Reference counts change by integer atomics, whose order does not show.  Moving
// pages is 16-byte streaming copies over the whole card.
//
// MI355X: the bookkeeping is a chain of dependent reads in one workgroup, 6 to 8 us a
// kernel over some ten thousand pages and rows that take a page or two.  What makes
// kv_page_reserve longer: one lane writes all new pages of its row, 0.18 us a page (a call
// that grows one row by 8192 tokens at pages of 16, 512 pages, 100 us, by 131072 tokens
// 1.43 ms; 32 rows by 500 to 8000 tokens 122 us, at pages of 64 38); and the free pages are
// looked for from page 1 on, 4096 a round (the lowest free one behind 2^17 others 60 us,
// behind 2^20 418).  Copying reads and writes at 5.0 TB/s (the rate of a large plain
// copy); packing 560 MB of pages takes 220 us behind 8 us of plan, 235 to 240 a call.

#include "attn_internal.h"
#include "device_common.h"

namespace gdn {

namespace {

constexpr int NT = 1024; // the bookkeeping workgroup
constexpr int CT = 256;  // a copying workgroup
constexpr int CV = 4;    // 16-byte pieces of a copying thread

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The sum of v over the workgroup's threads before this one; total: over all.
__device__ __forceinline__ int scan_exclusive(int v, int *total)
{
    __shared__ int wave_sum[NT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(inc, m);
        if (lane >= m)
            inc += o;
    }
    __syncthreads(); // the sums of the scan before are read
    if (lane == 63)
        wave_sum[wave] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        before += w < wave ? wave_sum[w] : 0;
        all += wave_sum[w];
    }
    *total = all;
    return before + inc - v;
}

__device__ __forceinline__ int pages_of(int len, int shift)
{
    return (int)(((int64_t)len + (1 << shift) - 1) >> shift);
}

// owner[r] = the first list entry that names row r, for every row that the list names.
__device__ __forceinline__ void first_owners(const PageParams &p, const int32_t *rows)
{
    for (int i = threadIdx.x; i < p.n; i += NT)
        if (rows[i] > 0 && rows[i] < p.R)
            __hip_atomic_store(&p.owner[rows[i]], p.n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += NT)
        if (rows[i] > 0 && rows[i] < p.R)
            atomicMin(&p.owner[rows[i]], i);
    __syncthreads();
}

__device__ __forceinline__ bool owns(const PageParams &p, int row, int i)
{
    return __hip_atomic_load(&p.owner[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == i;
}

// The numbers of the first `want` free pages, ascending, into list; how many there are of them.
__device__ __forceinline__ int list_free(const PageParams &p, int want, int32_t *list)
{
    int got = 0;
    for (int base = 0; base < p.N && got < want; base += 4 * NT) {
        const int id = base + 4 * (int)threadIdx.x;
        bool is_free[4];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            is_free[k] = id + k > 0 && id + k < p.N && p.refs[id + k] <= 0;
            mine += is_free[k];
        }
        int all;
        int at = got + scan_exclusive(mine, &all);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (is_free[k] && at < want) // at counts on past want
                list[at++] = id + k;
        got += all;
    }
    __syncthreads();
    return got < want ? got : want;
}


} // namespace

// plan: [n] the sum of needs before entry i, -1 for one that cannot be served;
// [n] fork: its length, -1 if not served; [2 n] fork: last page and its copy;
// then the free list (at most N).
__global__ __launch_bounds__(NT) void kv_reserve_kernel(PageParams p)
{
    __shared__ int missed, first;
    if (threadIdx.x == 0) {
        missed = 0;
        first = p.n;
    }
    int32_t *before = p.plan, *list = p.plan + 4 * (int64_t)p.n;
    const int top = p.width << p.page_shift;
    first_owners(p, p.a);
    int want = 0;
    for (int base = 0; base < p.n; base += NT) {
        const int i = base + threadIdx.x;
        bool ok = false;
        int need = 0;
        if (i < p.n) {
            const int r = p.a[i], add = p.b[i];
            if (r > 0 && r < p.R && owns(p, r, i)) {
                const int len = p.kv_len[r];
                ok = add >= 0 && len >= 0 && len <= top && add <= top - len;
                if (ok)
                    need = pages_of(len + add, p.page_shift) - pages_of(len, p.page_shift);
            }
        }
        int all;
        // a sum past the pool's size serves nobody: held there, so that it cannot overflow
        const int at = scan_exclusive(need < p.N ? need : p.N, &all);
        if (i < p.n)
            before[i] = ok ? want + at : -1;
        want = want + all < p.N ? want + all : p.N;
    }
    const int got = list_free(p, want, list);
    for (int i = threadIdx.x; i < p.n; i += NT) {
        bool served = before[i] >= 0;
        if (served) {
            const int r = p.a[i], len = p.kv_len[r], add = p.b[i];
            const int e0 = pages_of(len, p.page_shift), need = pages_of(len + add, p.page_shift) - e0;
            served = need == 0 || (need <= got && before[i] <= got - need);
            if (served) {
                for (int k = 0; k < need; ++k) {
                    const int page = list[before[i] + k];
                    p.table[(int64_t)r * p.width + e0 + k] = page;
                    p.refs[page] = 1;
                }
                p.kv_len[r] = len + add;
            }
        }
        if (!served) {
            atomicAdd(&missed, 1);
            atomicMin(&first, i);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.result[0] = missed;
        p.result[1] = missed ? first : -1;
    }
}

__global__ __launch_bounds__(NT) void kv_fork_plan_kernel(PageParams p)
{
    __shared__ int missed, first;
    if (threadIdx.x == 0) {
        missed = 0;
        first = p.n;
    }
    int32_t *before = p.plan, *length = p.plan + p.n, *from = p.plan + 2 * (int64_t)p.n,
            *to = p.plan + 3 * (int64_t)p.n, *list = p.plan + 4 * (int64_t)p.n;
    const int top = p.width << p.page_shift, inside = (1 << p.page_shift) - 1;
    first_owners(p, p.b);
    int want = 0;
    for (int base = 0; base < p.n; base += NT) {
        const int i = base + threadIdx.x;
        bool ok = false;
        int need = 0, len = -1;
        if (i < p.n) {
            const int src = p.a[i], dst = p.b[i];
            if (src > 0 && src < p.R && dst > 0 && dst < p.R && src != dst && owns(p, dst, i)) {
                len = p.kv_len[src];
                ok = len >= 0 && len <= top && p.kv_len[dst] == 0;
                need = ok && (len & inside) != 0;
            }
        }
        int all;
        const int at = scan_exclusive(need, &all);
        if (i < p.n) {
            before[i] = ok ? want + at : -1;
            length[i] = len;
        }
        want += all;
    }
    const int got = list_free(p, want < p.N ? want : p.N, list);
    // every source's length has been read: lengths may change now
    for (int i = threadIdx.x; i < p.n; i += NT) {
        const int len = length[i], need = (len & inside) != 0;
        const bool served = before[i] >= 0 && (!need || before[i] < got);
        from[i] = to[i] = 0;
        if (served) {
            const int dst = p.b[i];
            if (need) {
                const int e = len >> p.page_shift;
                const int old = p.table[(int64_t)p.a[i] * p.width + e], page = list[before[i]];
                p.table[(int64_t)dst * p.width + e] = page;
                p.refs[page] = 1;
                from[i] = old > 0 && old < p.N ? old : 0;
                to[i] = page;
            }
            p.kv_len[dst] = len;
        } else {
            length[i] = -1;
            atomicAdd(&missed, 1);
            atomicMin(&first, i);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        p.result[0] = missed;
        p.result[1] = missed ? first : -1;
    }
}

// One piece of a page of one layer's k or v: CT * CV 16-byte values.
__device__ __forceinline__ void copy_piece(const PageParams &p, int src, int dst, int64_t piece)
{
    const int64_t values = p.page_bytes / 16, pieces = (values + CT * CV - 1) / (CT * CV);
    const int64_t array = piece / pieces, at = (piece - array * pieces) * (CT * CV) + threadIdx.x;
    const int64_t layer = (array >> 1) * p.layer_stride;
    uint8_t *pages = ((array & 1) ? p.v : p.k) + layer;
    const u32x4 *s = reinterpret_cast<const u32x4 *>(pages + src * p.page_bytes);
    u32x4 *d = reinterpret_cast<u32x4 *>(pages + dst * p.page_bytes);
    u32x4 v[CV];
#pragma unroll
    for (int k = 0; k < CV; ++k)
        if (at + k * CT < values)
            v[k] = __builtin_nontemporal_load(s + at + k * CT);
#pragma unroll
    for (int k = 0; k < CV; ++k)
        if (at + k * CT < values)
            __builtin_nontemporal_store(v[k], d + at + k * CT);
}

static int64_t pieces_of(const PageParams &p)
{
    return 2 * (int64_t)p.layers * ((p.page_bytes / 16 + CT * CV - 1) / (CT * CV));
}

// blockIdx.y = entry: its whole pages are shared, its last page copied.
__global__ __launch_bounds__(CT) void kv_fork_share_kernel(PageParams p, int64_t pieces)
{
    const int i = blockIdx.y;
    const int len = p.plan[p.n + i];
    if (len < 0)
        return;
    const int32_t *src = p.table + (int64_t)p.a[i] * p.width;
    int32_t *dst = p.table + (int64_t)p.b[i] * p.width;
    for (int e = blockIdx.x * CT + threadIdx.x; e < len >> p.page_shift; e += gridDim.x * CT) {
        const int page = src[e];
        dst[e] = page;
        if (page > 0 && page < p.N)
            atomicAdd(&p.refs[page], 1);
    }
    const int from = p.plan[2 * (int64_t)p.n + i], to = p.plan[3 * (int64_t)p.n + i];
    if (from > 0 && to > 0)
        for (int64_t u = blockIdx.x; u < pieces; u += gridDim.x)
            copy_piece(p, from, to, u);
}

__global__ __launch_bounds__(CT) void kv_free_kernel(PageParams p)
{
    const int r = p.a[blockIdx.x];
    if (r <= 0 || r >= p.R)
        return;
    int32_t *row = p.table + (int64_t)r * p.width;
    for (int e = threadIdx.x; e < p.width; e += CT) {
        if (row[e] == 0)
            continue;
        const int page = atomicExch(&row[e], 0); // a row listed twice gives its pages back once
        if (page > 0 && page < p.N)
            atomicSub(&p.refs[page], 1);
    }
    if (threadIdx.x == 0)
        p.kv_len[r] = 0;
}

__global__ __launch_bounds__(CT) void kv_copy_kernel(PageParams p, int64_t pieces)
{
    const int64_t total = pieces * p.n;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int i = (int)(u / pieces);
        const int src = p.a[i], dst = p.b[i];
        if (dst > 0 && dst < p.N && src >= 0 && src < p.N)
            copy_piece(p, src, dst, u - i * pieces);
    }
}

// plan: [0] moves; then [N] sources and [N] destinations.
__global__ __launch_bounds__(NT) void kv_compact_plan_kernel(PageParams p)
{
    int32_t *src = p.plan + 1, *dst = src + p.N;
    int live = 0;
    for (int id = threadIdx.x; id < p.N; id += NT)
        live += id > 0 && p.refs[id] > 0;
    int m;
    scan_exclusive(live, &m);
    int ns = 0, nd = 0;
    for (int base = 0; base < p.N; base += NT) {
        const int id = base + (int)threadIdx.x;
        const bool on = id > 0 && id < p.N;
        const bool is_live = on && p.refs[id] > 0;
        const bool is_src = is_live && id > m, is_dst = on && !is_live && id <= m;
        int all;
        // two counts in one scan: at most 1024 of each a round
        const int at = scan_exclusive((is_src ? 1 : 0) + (is_dst ? 65536 : 0), &all);
        if (is_src)
            src[ns + (at & 65535)] = id;
        if (is_dst)
            dst[nd + (at >> 16)] = id;
        if (id < p.N)
            p.remap[id] = is_live ? id : 0;
        ns += all & 65535;
        nd += all >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < ns; k += NT) {
        const int a = src[k], b = dst[k];
        p.remap[a] = b;
        p.refs[b] = p.refs[a];
        p.refs[a] = 0;
    }
    if (threadIdx.x == 0) {
        p.plan[0] = ns;
        p.result[0] = m;
        p.result[1] = ns;
    }
}

__global__ __launch_bounds__(CT) void kv_compact_move_kernel(PageParams p, int64_t pieces)
{
    const int64_t entries = (int64_t)p.R * p.width;
    for (int64_t e = (int64_t)blockIdx.x * CT + threadIdx.x; e < entries; e += (int64_t)gridDim.x * CT) {
        const int page = p.table[e];
        if (page > 0 && page < p.N)
            p.table[e] = p.remap[page];
    }
    const int32_t *src = p.plan + 1, *dst = src + p.N;
    const int64_t total = pieces * p.plan[0];
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int i = (int)(u / pieces);
        copy_piece(p, src[i], dst[i], u - i * pieces);
    }
}

template <class... A>
static hipError_t launch(const void *f, dim3 grid, int threads, hipStream_t stream, A... a)
{
    void *args[] = {&a...};
    return hipLaunchKernel(f, grid, dim3(threads), args, 0, stream);
}

hipError_t launch_kv_reserve(const PageParams &p, hipStream_t stream)
{
    return launch(reinterpret_cast<const void *>(&kv_reserve_kernel), dim3(1), NT, stream, p);
}

hipError_t launch_kv_fork(const PageParams &p, hipStream_t stream)
{
    const hipError_t e = launch(reinterpret_cast<const void *>(&kv_fork_plan_kernel), dim3(1), NT, stream, p);
    if (e != hipSuccess || p.n == 0)
        return e;
    const int64_t pieces = pieces_of(p);
    return launch(reinterpret_cast<const void *>(&kv_fork_share_kernel),
                  dim3((unsigned)(pieces < 64 ? pieces : 64), (unsigned)p.n), CT, stream, p, pieces);
}

hipError_t launch_kv_free(const PageParams &p, hipStream_t stream)
{
    return launch(reinterpret_cast<const void *>(&kv_free_kernel), dim3((unsigned)p.n), CT, stream, p);
}

static unsigned copy_grid(int64_t total) { return (unsigned)(total < 65536 ? total : 65536); }

hipError_t launch_kv_copy(const PageParams &p, hipStream_t stream)
{
    const int64_t pieces = pieces_of(p);
    return launch(reinterpret_cast<const void *>(&kv_copy_kernel), dim3(copy_grid(pieces * p.n)), CT, stream, p,
                  pieces);
}

hipError_t launch_kv_compact(const PageParams &p, hipStream_t stream)
{
    const hipError_t e = launch(reinterpret_cast<const void *>(&kv_compact_plan_kernel), dim3(1), NT, stream, p);
    if (e != hipSuccess)
        return e;
    return launch(reinterpret_cast<const void *>(&kv_compact_move_kernel), dim3(4096), CT, stream, p, pieces_of(p));
}

} // namespace gdn
