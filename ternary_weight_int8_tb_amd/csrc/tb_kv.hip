// tb_kv.hip -- block tables and slots of a step, and rotary positions into the paged cache (gfx950).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tb.h"
#include "tb_heads.h"
#include "tb_rows.h"

namespace {

using namespace tbr;

// ------------------------------------------------------------------------------------
// The plan: one workgroup. Its parts depend on one another (rows cut at the step's, pages
// pushed before they are popped, slots read from the table's new entries), each is a scan over the
// requests or a few entries a thread, and up to hundreds of requests a second launch costs more than they do.
// Pages taken and rows of the step are dealt to the threads, not requests: their numbers differ by
// request from none to hundreds. A thread finds its request by a search in the scan, in LDS.
// Bound: latency, of some twenty dependent accesses. 1 request 5 us; 250 requests, 2048 rows 11; 2048 requests, 16384
// rows 28, most of which are the rows' lengths and table entries, read one behind the other, four rows a thread: positions and slots
// in a second launch over all CUs might take less there; not tried. (Four entries a thread with their loads in flight together: 8, 13 and 29.)
// ------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kMaxRequests = 16384;
constexpr int kMaxTokens = 1 << 30;

struct PlanArgs {
    const int32_t *context, *fresh;
    int requests, rows, page_shift, pages;
    int32_t *table;
    int width;
    int32_t *free_list;
    const int32_t *count;
    int32_t *lengths, *offsets, *positions, *slots, *left, *missing;
};

// Sum of v over the threads before this one, and over all. `cap` bounds every sum (all v are at most
// cap, and so are the results: min(sum, cap)).
__device__ __forceinline__ int block_scan(int v, int cap, int *wave_s, int *total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(sum, d);
        if (lane >= d)
            sum = min(sum + up, cap);
    }
    if (lane == 63)
        wave_s[wave] = sum;
    const int before = __shfl_up(sum, 1);
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        if (w == wave)
            base = all;
        all = min(all + wave_s[w], cap);
    }
    __syncthreads();   // wave_s is free again
    *total = all;
    return min(base + (lane ? before : 0), cap);
}

// The last i in [0, n) with at[i] <= x, where at[0] <= x, and at does not descend
__device__ __forceinline__ int last_up_to(const int *at, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(PlanArgs a)
{
    __shared__ int off_s[kMaxRequests + 1];    // rows before each request; before that, the ended requests
    __shared__ int page_s[kMaxRequests + 1];   // pages taken (or given back) before each
    __shared__ int wave_s[kPlanThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = a.requests, per = (n + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * per, n), r1 = min(r0 + per, n), page = 1 << a.page_shift;
    auto pages_of = [&](int tokens) { return min((int)(((unsigned)tokens + page - 1) >> a.page_shift), a.width); };
    auto context = [&](int r) { return min(max(a.context[r], 0), kMaxTokens); };

    // pages of ended requests go back
    int ended = 0, given = 0, total;
    for (int r = r0; r < r1; ++r)
        if (a.fresh[r] < 0) {
            ++ended;
            given += pages_of(context(r));
        }
    int all_ended, all_given = 0;
    int at = block_scan(ended, n, wave_s, &all_ended);
    int count = min(max(*a.count, 0), a.pages);
    if (all_ended) {
        int before = block_scan(given, INT32_MAX / 2, wave_s, &all_given);
        for (int r = r0; r < r1; ++r)
            if (a.fresh[r] < 0) {
                off_s[at] = r;
                page_s[at++] = before;
                before += pages_of(context(r));
            }
        __syncthreads();
        // A wave copies a request's entries; that all of them name pages is checked on the way.
        bool strange = false;
        for (int e = wave; e < all_ended; e += kPlanThreads / 64) {
            const int r = off_s[e], have = pages_of(context(r)), to = count + page_s[e];
            const int32_t *row = a.table + (size_t)r * a.width;
            for (int j = lane; j < have; j += 64) {
                const int id = row[j];
                strange |= (unsigned)id >= (unsigned)a.pages;
                if (to + j < a.pages)
                    a.free_list[to + j] = id;
            }
        }
        if (__syncthreads_or(strange)) {
            // entries to pass over: one wave, in order
            if (wave == 0) {
                int to = count;
                for (int e = 0; e < all_ended; ++e) {
                    const int r = off_s[e], have = pages_of(context(r));
                    const int32_t *row = a.table + (size_t)r * a.width;
                    for (int j0 = 0; j0 < have; j0 += 64) {
                        const int id = j0 + lane < have ? row[j0 + lane] : -1;
                        const bool good = (unsigned)id < (unsigned)a.pages;
                        const unsigned long long set = __ballot(good);
                        const int mine = to + __popcll(set & ((1ull << lane) - 1));
                        if (good && mine < a.pages)
                            a.free_list[mine] = id;
                        to += __popcll(set);
                    }
                }
                if (lane == 0)
                    wave_s[0] = to - count;
            }
            __syncthreads();
            all_given = wave_s[0];
        }
        __syncthreads();
        count = min((long long)count + all_given, (long long)a.pages);
    }

    // rows of the step, lengths, and the pages that they take
    int rows = 0;
    for (int r = r0; r < r1; ++r)
        rows = min(rows + min(max(a.fresh[r], 0), a.rows), a.rows);
    int row = block_scan(rows, a.rows, wave_s, &total);
    const int all_rows = total;
    int taken = 0;
    for (int r = r0, t = row; r < r1; ++r) {
        const int c = context(r), f = a.fresh[r], next = min(t + min(max(f, 0), a.rows), a.rows);
        off_s[r] = t;
        taken += max(pages_of(c + (next - t)) - pages_of(c), 0);
        t = next;
    }
    int before = block_scan(taken, INT32_MAX / 2, wave_s, &total);
    const int all_taken = total;
    for (int r = r0, t = row; r < r1; ++r) {
        const int c = context(r), f = a.fresh[r], next = min(t + min(max(f, 0), a.rows), a.rows);
        page_s[r] = before;
        before += max(pages_of(c + (next - t)) - pages_of(c), 0);
        a.offsets[r] = t;
        a.lengths[r] = f < 0 ? 0 : c + (next - t);   // context may be the same array: read before, by this thread
        t = next;
    }
    if (tid == 0) {
        off_s[n] = all_rows;
        page_s[n] = all_taken;
        a.offsets[n] = all_rows;
        *a.left = max(count - all_taken, 0);
    }
    __syncthreads();

    // new entries of the table. A request's first new page is the one behind its context's; the length
    // tells, as context may be gone.
    for (int i = tid; i < all_taken; i += kPlanThreads) {
        const int r = last_up_to(page_s, n + 1, i), new_pages = page_s[r + 1] - page_s[r];
        const int j = pages_of(a.lengths[r]) - new_pages + (i - page_s[r]), from = count - 1 - i;
        a.table[(size_t)r * a.width + j] = from >= 0 ? a.free_list[from] : -1;
    }
    __syncthreads();

    // positions and slots, four rows a thread
    int none = 0;
    for (int t0 = tid * 4; t0 < a.rows; t0 += kPlanThreads * 4) {
        int pos[4], slot[4];
        int r = t0 < all_rows ? last_up_to(off_s, n + 1, t0) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = t0 + e;
            pos[e] = slot[e] = -1;
            if (t < all_rows) {
                while (off_s[r + 1] <= t)   // off_s[n] = all_rows > t ends it
                    ++r;
                pos[e] = a.lengths[r] - (off_s[r + 1] - t);
                const int j = pos[e] >> a.page_shift;
                const int id = j < a.width ? a.table[(size_t)r * a.width + j] : -1;
                if ((unsigned)id < (unsigned)a.pages)
                    slot[e] = (id << a.page_shift) + (pos[e] & (page - 1));
                else
                    ++none;
            }
        }
        if (t0 + 4 <= a.rows) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int e = 0; t0 + e < a.rows; ++e) {
                a.positions[t0 + e] = pos[e];
                a.slots[t0 + e] = slot[e];
            }
        }
    }
    block_scan(none, INT32_MAX / 2, wave_s, &total);
    if (tid == 0)
        *a.missing = total;
}

// ------------------------------------------------------------------------------------
// Rotary positions. A workgroup takes a token's heads of q, k and v: its angles are made once, into
// LDS, and a thread turns 8 pairs at a time: 16 elements, which are two runs of 8 (half layout) or
// one of 16 (interleaved, or not turned at all). Bound: memory (8192 bf16 tokens of 16 + 2 + 2 heads of 256: 168 MB in 36 us,
// 4.6 TB/s; one token 3.9 us).
// The angle, in turns, is reduced in fp64 to a quarter: positions of any size keep it to 2^-24.
// ------------------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kMaxDim = 512;

struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    int tokens, dim, q_heads, kv_heads, rot, layout, dtype, cache_dtype, page_shift;
    uint32_t slots_end;
    float factor;
    const double *freq;
    const int32_t *positions, *slots;
    void *q_out;
    uint8_t *kc, *vc;
};

__device__ __forceinline__ void store8(void *p, size_t at, int dtype, const float *v)
{
    const float(&w)[8] = *reinterpret_cast<const float(*)[8]>(v);
    if (dtype == TB_F32) {
        Eight<float> e;
        e.set(w);
        e.store(static_cast<float *>(p) + at);
    } else if (dtype == TB_BF16) {
        Eight<Bf16> e;
        e.set(w);
        e.store(static_cast<Bf16 *>(p) + at);
    } else {
        Eight<F16> e;
        e.set(w);
        e.store(static_cast<F16 *>(p) + at);
    }
}

template <class T>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a)
{
    __shared__ float cos_s[kMaxDim / 2], sin_s[kMaxDim / 2];
    const int tid = threadIdx.x, t = blockIdx.x;
    const int p = a.positions[t];
    if (p < 0)
        return;
    for (int i = tid; i < a.rot / 2; i += kRopeThreads) {
        const double quarters = (double)p * a.freq[i] * 0.63661977236758134308;   // 2 / pi
        const double whole = rint(quarters);
        const int quarter = (int)(whole - 4.0 * floor(whole * 0.25));   // whole is exact, and so is this
        float s, c;
        sincospif((float)(quarters - whole) * 0.5f, &s, &c);
        const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
        cos_s[i] = a.factor * (quarter == 1 || quarter == 2 ? -x : x);
        sin_s[i] = a.factor * (quarter >= 2 ? -y : y);
    }
    __syncthreads();
    const int per_head = a.dim / 16, turned = a.rot / 16;
    const uint32_t slot = a.kv_heads ? (uint32_t)a.slots[t] : 0u;
    const bool cached = a.kv_heads && slot < a.slots_end;
    const int items = (a.q_heads + (cached ? 2 * a.kv_heads : 0)) * per_head;
    for (int item = tid; item < items; item += kRopeThreads) {
        const int head = item / per_head, c = item - head * per_head;
        // 0: q, 1: k, 2: v
        const int kind = head < a.q_heads ? 0 : head < a.q_heads + a.kv_heads ? 1 : 2;
        const int h = kind == 0 ? head : kind == 1 ? head - a.q_heads : head - a.q_heads - a.kv_heads;
        const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + t * (kind == 0 ? a.q_row : kind == 1 ? a.k_row : a.v_row) +
                       h * (kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head);
        const bool turn = kind < 2 && c < turned;
        const bool apart = turn && a.layout == TB_ROPE_HALF;
        const int lo = apart ? 8 * c : 16 * c, hi = apart ? a.rot / 2 + 8 * c : 16 * c + 8;
        Eight<T> el, eh;
        el.load(src + lo);
        eh.load(src + hi);
        float x[16], y[16];
        el.get(*reinterpret_cast<float(*)[8]>(x));
        eh.get(*reinterpret_cast<float(*)[8]>(x + 8));
        if (turn) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float cs = cos_s[8 * c + e], sn = sin_s[8 * c + e];
                // half: pairs (x[e], x[8 + e]); interleaved: (x[2 e], x[2 e + 1])
                const float u = apart ? x[e] : x[2 * e], w = apart ? x[8 + e] : x[2 * e + 1];
                const float ru = u * cs - w * sn, rw = w * cs + u * sn;
                if (apart)
                    y[e] = ru, y[8 + e] = rw;
                else
                    y[2 * e] = ru, y[2 * e + 1] = rw;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                y[e] = x[e];
        }
        if (kind == 0) {
            const size_t at = ((size_t)t * a.q_heads + h) * a.dim;
            store8(a.q_out, at + lo, a.dtype, y);
            store8(a.q_out, at + hi, a.dtype, y + 8);
        } else {
            const size_t page = slot >> a.page_shift, place = slot & ((1u << a.page_shift) - 1);
            const size_t at = (((page * a.kv_heads + h) << a.page_shift) + place) * a.dim;
            uint8_t *cache = kind == 1 ? a.kc : a.vc;
            store8(cache, at + lo, a.cache_dtype, y);
            store8(cache, at + hi, a.cache_dtype, y + 8);
        }
    }
}

}  // namespace

extern "C" int tb_kv_plan(const int32_t *context, const int32_t *fresh, int requests, int rows, int page, int pages, int32_t *table,
                          int width, int32_t *free_list, const int32_t *count, int32_t *lengths, int32_t *offsets,
                          int32_t *positions, int32_t *slots, int32_t *left, int32_t *missing, void *stream)
{
    if (requests < 1 || rows < 1 || width < 1 || pages < 1 || !tbh::page_ok(page) || (long long)pages * page >= (1ll << 31))
        return TB_EINVAL;
    const size_t r = (size_t)requests * 4, t = (size_t)rows * 4;
    // lengths may be context and left may be count: the one workgroup reads them before it writes there
    tbh::Arg a[11] = {{context, r, lengths == context},
                      {fresh, r, false},
                      {table, r * (size_t)width, true},
                      {free_list, (size_t)pages * 4, true},
                      {count, 4, left == count},
                      {offsets, r + 4, true},
                      {positions, t, true},
                      {slots, t, true},
                      {missing, 4, true}};
    size_t n = 9;
    if (lengths != context)
        a[n++] = {lengths, r, true};
    if (left != count)
        a[n++] = {left, 4, true};
    if (int rc = tbh::check_args(a, n))
        return rc;
    if (requests > kMaxRequests || rows >= kMaxTokens || (long long)requests * width >= kMaxTokens || (long long)width * page > kMaxTokens)
        return TB_EUNSUPPORTED;
    const PlanArgs p{context, fresh, requests, rows, tbh::log2_of(page), pages, table, width, free_list, count,
                     lengths, offsets, positions, slots, left, missing};
    hipLaunchKernelGGL(kv_plan_kernel, dim3(1), dim3(kPlanThreads), 0, static_cast<hipStream_t>(stream), p);
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

extern "C" int tb_rope_kv(const tb_heads *q, const tb_heads *k, const tb_heads *v, int tokens, int dim, const tb_rope *rope,
                          const int32_t *positions, const int32_t *slots, const tb_kv_cache *cache, void *q_out, int dtype,
                          void *stream)
{
    const bool kv = k || v || slots || cache;
    if (tokens < 1 || dim < 16 || dim > kMaxDim || dim % 16 || (!q && !kv) || !q != !q_out || (kv && !(k && v && slots && cache)))
        return TB_EINVAL;
    if (rope && (rope->rot < 16 || rope->rot > dim || rope->rot % 16 || (rope->layout != TB_ROPE_HALF && rope->layout != TB_ROPE_INTERLEAVED)))
        return TB_EINVAL;
    tbh::Arg a[9];
    size_t n = 0;
    a[n++] = {positions, (size_t)tokens * 4, false};
    if (rope)
        a[n++] = {rope->freq, (size_t)rope->rot * 4, false};
    const int rows_dtype = q ? q->dtype : k->dtype;
    for (const tb_heads *h : {q, k, v}) {
        if (!h)
            continue;
        const size_t bytes = tbh::heads_bytes(*h, tokens, dim);
        if (!bytes || h->dtype != rows_dtype)
            return TB_EINVAL;
        a[n++] = {h->data, bytes, false};
    }
    if (q) {
        if (!tbh::dtype_bytes(dtype))
            return TB_EINVAL;
        a[n++] = {q_out, (size_t)tokens * (size_t)q->heads * (size_t)dim * tbh::dtype_bytes(dtype), true};
    }
    if (kv) {
        if (!tbh::cache_ok(*cache) || cache->dim != dim || k->heads != cache->kv_heads || v->heads != cache->kv_heads)
            return TB_EINVAL;
        a[n++] = {slots, (size_t)tokens * 4, false};
        a[n++] = {cache->k, tbh::cache_bytes(*cache), true};
        a[n++] = {cache->v, tbh::cache_bytes(*cache), true};
    }
    if (int rc = tbh::check_args(a, n))
        return rc;
    if (tokens >= (1 << 24))   // 256 threads each, in 32 bits
        return TB_EUNSUPPORTED;
    RopeArgs r{};
    if (q)
        r.q = q->data, r.q_row = q->row_stride, r.q_head = q->head_stride, r.q_heads = q->heads, r.q_out = q_out, r.dtype = dtype;
    if (kv) {
        r.k = k->data, r.k_row = k->row_stride, r.k_head = k->head_stride;
        r.v = v->data, r.v_row = v->row_stride, r.v_head = v->head_stride;
        r.kv_heads = cache->kv_heads, r.cache_dtype = cache->dtype, r.page_shift = tbh::log2_of(cache->page);
        r.slots_end = (uint32_t)cache->pages << r.page_shift, r.slots = slots;
        r.kc = static_cast<uint8_t *>(cache->k), r.vc = static_cast<uint8_t *>(cache->v);
    }
    if (rope)
        r.rot = rope->rot, r.layout = rope->layout, r.factor = rope->factor, r.freq = rope->freq;
    r.tokens = tokens, r.dim = dim, r.positions = positions;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid(tokens), block(kRopeThreads);
    switch (rows_dtype) {
    case TB_F32: hipLaunchKernelGGL(rope_kernel<float>, grid, block, 0, st, r); break;
    case TB_BF16: hipLaunchKernelGGL(rope_kernel<Bf16>, grid, block, 0, st, r); break;
    default: hipLaunchKernelGGL(rope_kernel<F16>, grid, block, 0, st, r); break;
    }
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}
