// tb_attn.hip -- attention of the newest tokens over a paged cache (gfx950).
//
//   o = sum_j softmax_j(scale q . k_j) v_j,  out = o / (1 + exp(-gate))
//
// One pass over the keys with a running maximum and sum for each row. Rows of a request are its (token,
// head) pairs that share a kv head: row r is token r / group, head r % group. A unit is a tile of
// such rows with all the keys that any of them sees; the units of a call, counted in steps of a fixed
// number of keys, are dealt to the workgroups in equal stretches, whatever the requests' lengths
// are, and a second launch joins the units that a border cuts.
//
// Both products are transposed, with the rows as columns of the 16 x 16 x 32 matrix instruction:
// S^T = K Q^T and O^T = V^T P^T. A lane then holds scores of one row only, its maximum and
// factors are the lane's own, and its 8 weights of 32 keys are an operand of the second product as they
// stand: the order of the 32 keys is free, as long as V^T's columns have the same one.
// V^T comes from rows of V in LDS by transposing reads (ds_read_b64_tr_b16).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tb.h"
#include "tb_heads.h"
#include "tb_rows.h"

namespace {

using namespace tbr;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_t;
typedef const __attribute__((address_space(4))) int32_t *const_ints;   // read by scalar loads

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kBlk = 32;   // keys of a matrix step

struct AttnArgs {
    const void *q, *gate;
    int64_t q_row, q_head, g_row, g_head;
    int gate_dtype;
    const uint8_t *k, *v;
    const int32_t *table, *offsets, *lengths;
    int pages, page_shift, width, kv_heads, group, requests, tokens, window;
    uint32_t group_mul, group_shift;   // x / group = (x + mulhi(x, mul)) >> shift, for x < 2^31
    float scale;   // times log2(e)
    void *out;
    int32_t *meta;
    float *part;
};

// ---- types of the products ----------------------------------------------------------
__device__ __forceinline__ v4f mfma(uint4 a, uint4 b, v4f c, Bf16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(uint4 a, uint4 b, v4f c, F16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
// c + the sum of the products of two pairs
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c, Bf16)
{
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), __builtin_bit_cast(b2, b), c, false);
}
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c, F16)
{
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
}
__device__ __forceinline__ constexpr uint32_t ones(Bf16) { return 0x3f803f80u; }
__device__ __forceinline__ constexpr uint32_t ones(F16) { return 0x3c003c00u; }
// bits of the exponent in a pair
__device__ __forceinline__ constexpr uint32_t exponents(Bf16) { return 0x7f807f80u; }
__device__ __forceinline__ constexpr uint32_t exponents(F16) { return 0x7c007c00u; }

// fp32 values as parts in T whose sum has 24 bits (bf16: three parts, each cut off, not rounded, so that
// the rest is exact) or 22 (fp16: two, as far as the second is above 2^-14: below it is off by 2^-25). One part: rounded to nearest.
template <class T, bool EXACT>
struct Split {
    static constexpr int kParts = 1;
    static __device__ __forceinline__ void pair(float a, float b, uint32_t (&w)[1]) { w[0] = pack(a, b, T()); }
};
template <>
struct Split<Bf16, true> {
    static constexpr int kParts = 3;
    static __device__ __forceinline__ void pair(float a, float b, uint32_t (&w)[3])
    {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
            w[p] = __builtin_amdgcn_perm(ub, ua, 0x07060302);
            a -= __uint_as_float(ua & 0xffff0000u);
            b -= __uint_as_float(ub & 0xffff0000u);
        }
    }
};
template <>
struct Split<F16, true> {
    static constexpr int kParts = 2;
    static __device__ __forceinline__ void pair(float a, float b, uint32_t (&w)[2])
    {
        w[0] = pack(a, b, F16());
        float ha, hb;
        unpack(w[0], ha, hb, F16());
        w[1] = pack(a - ha, b - hb, F16());
    }
};
// The larger of two scores, in one operation: fmaxf first makes each operand, which the matrix instruction has written, a quiet
// number, in one each, and the compiler makes fmaxf of a median whose third number it knows. (With a NaN the other, with two
// infinity: such a row has no result anyway.)
__device__ __forceinline__ float larger(float a, float b)
{
    float inf = INFINITY;
    asm("" : "+s"(inf));
    return __builtin_amdgcn_fmed3f(a, b, inf);
}

__device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// v, of which the compiler does not know that it is v: what is derived from it is derived where it is used, and not kept in
// registers from before the loops
__device__ __forceinline__ int opaque(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// What few blocks of keys meet: its code stands apart, and the others' together (2048 behind 8192: 313 -> 303 us)
__device__ __forceinline__ bool rarely(bool v) { return __builtin_expect(v, 0); }

__device__ __forceinline__ int by_group(const AttnArgs &a, int x)
{
    return (int)((__umulhi((uint32_t)x, a.group_mul) + (uint32_t)x) >> a.group_shift);
}

// ---- units --------------------------------------------------------------------------
struct Unit {
    int first, n, len;   // the request's first row of q, its new tokens, its length
    int tile;
    int kbeg, kend;      // keys that any of its rows sees
    int s0, steps;       // its first step, in steps from key 0 on, and their number (one at least)
    int cost;            // what it takes on the line of units: its steps, and what beginning and ending it takes, in steps
};

__device__ __forceinline__ void request_of(const AttnArgs &a, int r, int &first, int &n, int &len)
{
    first = min(max(a.offsets[r], 0), a.tokens);
    n = min(max(a.offsets[r + 1], first), a.tokens) - first;
    len = min(max(a.lengths[r], 0), 1 << 30);
}
// Offsets that descend give rows to several requests, and a line of units longer than the host has checked: such a call does nothing.
__device__ __forceinline__ bool descends(const AttnArgs &a, int r)
{
    return min(max(a.offsets[r + 1], 0), a.tokens) < min(max(a.offsets[r], 0), a.tokens);
}
template <int ROWS>
__device__ __forceinline__ int tiles_of(const AttnArgs &a, int n)
{
    return (n * a.group + ROWS - 1) / ROWS;
}
template <int ROWS, int STEP, int EXTRA>
__device__ __forceinline__ void span(const AttnArgs &a, Unit &u)
{
    const int r0 = u.tile * ROWS, r1 = min(r0 + ROWS, u.n * a.group) - 1;
    const int p0 = u.len - u.n + by_group(a, r0), p1 = u.len - u.n + by_group(a, r1);
    u.kend = max(min(min(u.len, a.width << a.page_shift), p1 + 1), 0);
    u.kbeg = a.window ? min(max(p0 - a.window + 1, 0), u.kend) : 0;
    u.s0 = u.kbeg / STEP;
    u.steps = max((u.kend + STEP - 1) / STEP - u.s0, 1);
    u.cost = u.steps + EXTRA;
}

// Sum over the threads before this one, and over all.
template <int WAVES>
__device__ __forceinline__ int scan(int v, int *wave_s, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(sum, d);
        sum += lane >= d ? up : 0;
    }
    __syncthreads();
    if (lane == 63)
        wave_s[wave] = sum;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        base += w < wave ? wave_s[w] : 0;
        total += wave_s[w];
    }
    return base + sum - v;
}

struct Start {
    int all;             // cost of all units of a kv head
    int req, into;       // the unit where the slot's stretch of the line begins, and the line's place in it
    Unit u;
};

// A thread's walk along the tiles of the requests.
template <int ROWS, int STEP, int EXTRA>
struct Walk {
    int r, left;   // the request, and its tiles from the current one on
    Unit u;
    __device__ __forceinline__ void open(const AttnArgs &a)
    {
        request_of(a, r, u.first, u.n, u.len);
        left = tiles_of<ROWS>(a, u.n);
        u.tile = 0;
    }
    __device__ __forceinline__ void next(const AttnArgs &a)
    {
        ++u.tile;
        if (--left == 0) {
            while (++r < a.requests) {
                open(a);
                if (left)
                    break;
            }
        }
    }
};

// Every workgroup lays the whole line of units out for itself: a few thousand of them at most, a handful per
// thread, which is less than a launch for a plan would take.
template <int ROWS, int STEP, int EXTRA, int WAVES>
__device__ __forceinline__ void find_start(const AttnArgs &a, int slots, int slot, int *chunk_s, int *wave_s, int *found_s, Start &st, unsigned &per)
{
    using W = Walk<ROWS, STEP, EXTRA>;
    // the host has checked that the whole line is shorter than 2^31
    auto share_of = [&](int all) { return max(((unsigned)all * (unsigned)a.kv_heads + (unsigned)slots - 1u) / (unsigned)slots, 1u); };
    if (a.requests <= 64 && a.tokens <= a.requests) {
        // a token for each request at most, as in decoding: a wave looks at them alone
        const int lane = threadIdx.x & 63;
        W w;
        w.r = lane;
        int cost = 0;
        if (__any(lane < a.requests && descends(a, lane))) {
            st.all = 0;
            per = 1;
            return;
        }
        if (lane < a.requests) {
            w.open(a);
            while (w.r == lane && w.left) {
                span<ROWS, STEP, EXTRA>(a, w.u);
                cost += w.u.cost;
                ++w.u.tile, --w.left;
            }
        }
        int sum = cost;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            sum += lane >= d ? up : 0;
        }
        st.all = __builtin_amdgcn_readlane(sum, 63);
        per = share_of(st.all);
        if (st.all == 0)
            return;
        const int want = (int)((unsigned)slot * per % (unsigned)st.all);
        const int at = __builtin_ctzll(__ballot(sum > want));   // the request: want < st.all
        st.req = at;
        st.into = want - __builtin_amdgcn_readlane(sum - cost, at);
        w.r = at;
        w.open(a);
        for (;; ++w.u.tile) {
            span<ROWS, STEP, EXTRA>(a, w.u);
            if (st.into < w.u.cost || --w.left == 0)
                break;
            st.into -= w.u.cost;
        }
        st.into = __builtin_amdgcn_readfirstlane(st.into);
        st.u = {__builtin_amdgcn_readfirstlane(w.u.first), __builtin_amdgcn_readfirstlane(w.u.n), __builtin_amdgcn_readfirstlane(w.u.len),
                __builtin_amdgcn_readfirstlane(w.u.tile)};
        return;
    }
    constexpr int kThreads = WAVES * 64;
    const int tid = threadIdx.x, chunk = (a.requests + kThreads - 1) / kThreads;
    const int q0 = min(tid * chunk, a.requests), q1 = min(q0 + chunk, a.requests);
    int tiles = 0, first, n, len, total;
    bool none = false;
    for (int r = q0; r < q1; ++r) {
        request_of(a, r, first, n, len);
        tiles += tiles_of<ROWS>(a, n);
        none |= descends(a, r);
    }
    const int before = scan<WAVES>(none ? 0 : tiles, wave_s, total);
    chunk_s[tid] = before;
    if (__syncthreads_or(none)) {
        st.all = 0;
        per = 1;
        return;
    }
    const int share = (total + kThreads - 1) / kThreads, t0 = min(tid * share, total), t1 = min(t0 + share, total);
    // the chunk, then the request, of tile t0
    W w;
    auto locate = [&]() {
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_s[mid] <= t0)
                lo = mid;
            else
                hi = mid;
        }
        int t = t0 - chunk_s[lo];
        for (w.r = lo * chunk;; ++w.r) {   // t0 < total: the chunk holds it
            w.open(a);
            if (t < w.left || w.r + 1 >= a.requests)
                break;
            t -= w.left;
        }
        w.u.tile = t;
        w.left -= t;
    };
    int cost = 0;
    if (t0 < t1) {
        locate();
        for (int t = t0; t < t1; ++t) {
            span<ROWS, STEP, EXTRA>(a, w.u);
            cost += w.u.cost;
            if (t + 1 < t1)
                w.next(a);
        }
    }
    int at = scan<WAVES>(cost, wave_s, st.all);
    per = share_of(st.all);
    if (st.all == 0)
        return;
    const int want = (int)((unsigned)slot * per % (unsigned)st.all);
    if (t0 < t1 && at <= want && want < at + cost) {
        locate();
        for (int t = t0; t < t1; ++t) {
            span<ROWS, STEP, EXTRA>(a, w.u);
            if (want < at + w.u.cost)
                break;
            at += w.u.cost;
            w.next(a);
        }
        const int found[6] = {w.r, want - at, w.u.first, w.u.n, w.u.len, w.u.tile};
#pragma unroll
        for (int x = 0; x < 6; ++x)
            found_s[x] = found[x];
    }
    __syncthreads();
    st.req = __builtin_amdgcn_readfirstlane(found_s[0]);
    st.into = __builtin_amdgcn_readfirstlane(found_s[1]);
    st.u = {__builtin_amdgcn_readfirstlane(found_s[2]), __builtin_amdgcn_readfirstlane(found_s[3]), __builtin_amdgcn_readfirstlane(found_s[4]),
            __builtin_amdgcn_readfirstlane(found_s[5])};
}

// ---- a wave's rows ------------------------------------------------------------------
// Where 16 rows of K or V lie in LDS, so that neither the reads of K (16 rows of 16 bytes, 8 lanes a cycle) nor those of V
// (16 rows of 32 bytes) meet in the same banks (64 of 4 bytes).
//   D = 256: rows r and r + 8 side by side, which one load fills, and 32 bytes between such pairs: all places of a lane
//   are one register and constants.
//   Else four or eight rows side by side, and segment c of 32 bytes of row r at segment c ^ fold(r) of 8 or 4.
template <int D>
struct Lay {
    static constexpr bool kApart = D == 256;
    static constexpr int kPair = 1024 + 32, kGroup = kApart ? 8 * kPair : 16 * D * 2;
    static constexpr int kSegs = D >= 128 ? 8 : 4;                  // that fold turns
    static constexpr int kKinds = kApart ? 1 : kSegs;               // registers for a lane's places in V, and twice those in K
    static __device__ __forceinline__ int fold(int row) { return kApart ? 0 : D == 128 ? row & 7 : (row >> 1) & 3; }
    static __device__ __forceinline__ int row(int r) { return kApart ? (r & 7) * kPair + (r >> 3) * 512 : r * D * 2; }
};

// The same in all lanes, in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p)
{
    const uint64_t v = (uint64_t)p;
    return (const uint8_t *)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                             (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// 16 keys, one contiguous stretch of a page, to LDS
template <int D>
struct Loader {
    using L = Lay<D>;
    static constexpr int kLoads = D / 32;    // of 1 KB
    uint32_t off;                            // of the lane's 16 bytes in a load
    __device__ __forceinline__ void init(int lane)
    {
        constexpr int kLanes = D / 8;   // of a row
        const int row = lane / kLanes, c = lane % kLanes;
        off = L::kApart ? (uint32_t)(row * 8 * 512 + c * 16) : (uint32_t)(row * D * 2 + (((c >> 1) ^ L::fold(row)) << 5) + (c & 1) * 16);
    }
    __device__ __forceinline__ void pin() { asm volatile("" : "+v"(off)); }   // as Rows::pin_reads
    // `from` and `to` are the same in all lanes; lane l's 16 bytes go to to + 16 l. The compiler knows of the load's
    // writes to LDS, but not when they are done: for the builtin it waits for all loads at the next read of
    // any of it by ordinary loads, and never for transposing reads. So this is an asm without outputs, and each
    // read of a buffer stands behind a wait of its own (landed()).
    __device__ __forceinline__ void load(const uint8_t *from, lds_t *to) const
    {
        from = uniform(from);
        const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)to);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            // rows i and i + 8; or the next four or eight, whose fold differs from the first ones' in these bits alone
            const uint32_t turn = L::kApart ? 0u : (uint32_t)L::fold(i * (512 / D)) << 5;
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                         ::"s"(lds + i * (L::kApart ? L::kPair : 1024)), "v"(off ^ turn), "s"(from + i * (L::kApart ? 512 : 1024))
                         : "memory");   // m0 is the compiler's to set, and it sets it wherever it needs it
        }
    }
};
// Waits until at most N of the wave's loads are on their way: all but the N last ones have landed.
template <int N>
__device__ __forceinline__ void landed()
{
    static_assert(N >= 0 && N < 64, "six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The wave's reads of LDS are done.
__device__ __forceinline__ void lds_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// NT column tiles of 16 rows; lane l has, of each, row l % 16.
// AHEAD: operands of a block's first product are read together, and those of the second before the weights are made; else they
// come a few at a time, for want of registers.
template <int D, class T, bool EXACT, int NT, bool AHEAD>
struct Rows {
    static constexpr int kQ = D / 32, kO = D / 16, kParts = Split<T, EXACT>::kParts;
    // Weights start at 2^kBias (of fp32 rows at kUnit, a factor: in the exponent it would cost bits), and a row's maximum lags by a
    // factor of 2^kLag at most.
    // bf16: so far below one that sums of the largest values that the cache holds are fp32 numbers (of 2^20 keys, with weights up
    // to 2^-20), and no further, as fp32 ends at 2^-149: values down to 2^-110 keep their 8 bits under the largest weight.
    // fp16: so far above one that small weights keep their bits, and the largest, 2^14 or 2^15, still fits. Of fp32 rows a weight's
    // second part must keep its bits too. Its last one is 2^-24: both parts are off by 2^-25 at most, 2^-38 of the largest weight, and
    // the sum of 22 bits is whole from 2^-15 of that on. (At 2^6 weights of e^-16 would be off by up to 2^-8 of themselves.)
    static constexpr bool kFine = EXACT && std::is_same<T, F16>::value;
    static constexpr float kBias = std::is_same<T, F16>::value ? 6.0f : -28.0f, kUnit = kFine ? 0x1p13f : 0x1p-28f;
    static constexpr float kLag = kFine ? 2.0f : 8.0f;
    uint4 q[NT][kQ][kParts];
    v4f o[NT][kO];
    float m[NT], l[NT], factor[NT];   // running maximum of the scores, sum of the lane's weights, the scores' factor
    int pos[NT];                      // the row's position: it sees the keys up to it
    bool small;                       // all maxima are below kFused: see weigh()
    using L = Lay<D>;
    static constexpr int kKk = L::kApart ? 1 : L::kKinds / 2;
    uint32_t kread[kKk], vread[L::kKinds];   // the lane's places in a row of K, and of V

    // one factor for all rows, unless they have been scaled
    __device__ __forceinline__ float c(const AttnArgs &a, int n) const { return kFine ? factor[n] : a.scale; }

    __device__ __forceinline__ void init_reads(int lane)
    {
        const int i = lane & 15, g = lane >> 4, row = 4 * g + (i >> 2);
#pragma unroll
        for (int x = 0; x < kKk; ++x)
            kread[x] = (uint32_t)(L::row(i) + (((2 * x + (g >> 1)) ^ L::fold(i)) << 5) + (g & 1) * 16);
#pragma unroll
        for (int x = 0; x < L::kKinds; ++x)
            vread[x] = (uint32_t)(L::row(row) + ((x ^ L::fold(row)) << 5) + (i & 3) * 8);
    }
    // 16 keys' elements 32 s + 8 g .. + 7 of group t
    __device__ __forceinline__ uint4 key(const lds_t *buf, int t, int s) const
    {
        const uint32_t at = kread[s % kKk] + s / kKk * (L::kApart ? 64 : L::kSegs * 32);
        return __builtin_bit_cast(uint4, *(const __attribute__((address_space(3))) v4u *)(buf + at + t * L::kGroup));
    }
    // elements 16 d + lane % 16 of keys 4 g .. + 3 of both groups
    __device__ __forceinline__ uint4 value(const lds_t *buf, int d) const
    {
        const uint32_t at = vread[d % L::kKinds] + d / L::kKinds * (L::kApart ? 32 : L::kSegs * 32);
        uint2 w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            w[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(buf + at + t * L::kGroup)));
        return make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    }

    // Rows row0 .. row0 + 16 NT - 1 of a unit (rows past the last are that one): what they see, and their q, asked for
    // here and made operands by begin().
    struct Raw {
        Eight<typename std::conditional<EXACT, float, T>::type> e[NT][kQ];
    };
    __device__ __forceinline__ void fetch(const AttnArgs &a, const Unit &u, int head, int row0, int lane, Raw &raw)
    {
        using E = typename std::conditional<EXACT, float, T>::type;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = min(row0 + 16 * n + (lane & 15), u.n * a.group - 1), tok = by_group(a, r), h = head * a.group + r - tok * a.group;
            pos[n] = u.len - u.n + tok;
            const E *at = static_cast<const E *>(a.q) + (long long)(u.first + tok) * a.q_row + (long long)h * a.q_head + 8 * (lane >> 4);
#pragma unroll
            for (int s = 0; s < kQ; ++s)
                raw.e[n][s].load(at + 32 * s);
        }
    }
    __device__ __forceinline__ void begin(const AttnArgs &a, Raw &raw)
    {
        small = true;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (!EXACT) {
#pragma unroll
                for (int s = 0; s < kQ; ++s)
                    q[n][s][0] = raw.e[n][s].w;
            } else {
                split_q(a, n, raw.e[n]);
            }
            // loaded here, or the wait for these loads stands in the loop over the keys, where it would also be one for theirs
#pragma unroll
            for (int s = 0; s < kQ; ++s)
#pragma unroll
                for (int x = 0; x < kParts; ++x)
                    asm volatile("" : "+v"(q[n][s][x].x), "+v"(q[n][s][x].y), "+v"(q[n][s][x].z), "+v"(q[n][s][x].w));
            m[n] = -INFINITY;
            l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < kO; ++d)
                o[n][d] = v4f{};
        }
    }
    __device__ __forceinline__ void split_q(const AttnArgs &a, int n, Eight<float> (&e)[kQ])
    {
        if constexpr (std::is_same<T, F16>::value) {
            // the row's largest element between 2^9 and 2^10: whatever the row's magnitude, its parts are fp16 numbers
            float top = 0.0f, v[8];
#pragma unroll
            for (int s = 0; s < kQ; ++s) {
                e[s].get(v);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    top = fmaxf(top, fabsf(v[x]));
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int ex = top > 0.0f && top < INFINITY ? min(max((int)(__float_as_uint(top) >> 23), 1), 254) - 127 : 9;
            // 2^(9 - ex) in two factors, either of which fp32 holds
            const int half = (9 - ex) / 2;
            const float f = __builtin_ldexpf(1.0f, half), f2 = __builtin_ldexpf(1.0f, 9 - ex - half);
#pragma unroll
            for (int s = 0; s < kQ; ++s) {
                e[s].get(v);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    v[x] = v[x] * f * f2;
                e[s].set(v);
            }
            // Not 0 and not infinite, whose products with hidden scores and with the maximum's own difference are NaN. (Scores are
            // below 2^35, and their differences above 2^-50: beyond these limits all weights are alike, or one is all.)
            factor[n] = fminf(fmaxf(a.scale / f / f2, 0x1p-126f), 0x1.fffffep127f);
        }
#pragma unroll
        for (int s = 0; s < kQ; ++s) {
            float v[8];
            e[s].get(v);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t w[kParts];
                Split<T, EXACT>::pair(v[2 * x], v[2 * x + 1], w);
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    word(q[n][s][p], x) = w[p];
            }
        }
    }

    // Scores of 32 keys: s[n][t][i] is key 16 t + 4 g + i. Operands in batches, one on its way while the other is
    // multiplied.
    __device__ __forceinline__ void scores(const lds_t *kb, v4f (&s)[NT][2]) const
    {
        constexpr int kBatch = AHEAD ? 2 * kQ : NT > 1 ? 2 : 4, kBatches = 2 * kQ / kBatch;
        uint4 k[AHEAD ? 1 : 2][kBatch];
        auto read = [&](int b) {
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
                k[AHEAD ? 0 : b & 1][x] = key(kb, x & 1, (b * kBatch + x) >> 1);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n)
            s[n][0] = s[n][1] = v4f{};
        read(0);
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
            if (b + 1 < kBatches)
                read(b + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = kParts; p-- > 0;)
#pragma unroll
                for (int x = 0; x < kBatch; ++x)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        s[n][x & 1] = mfma(k[AHEAD ? 0 : b & 1][x], q[n][(b * kBatch + x) >> 1][p], s[n][x & 1], T());
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Does row n see key k? (Keys from a unit's kend on are seen by none: their values are zeros, and see hide().)
    __device__ __forceinline__ bool sees(const AttnArgs &a, int n, int k) const { return k <= pos[n] && (!a.window || k > pos[n] - a.window); }
    // Scores of keys that a row does not see. `there`: bit x set where key x of the 32 is one that some row of the unit sees.
    // (A mask of the lane's eight keys for each tile of rows, and fences: the loop over the keys has no registers to spare.)
    __device__ __forceinline__ void hide(const AttnArgs &a, int key0, int lane, uint32_t there, v4f (&s)[NT][2]) const
    {
        const int first = lane >> 4 << 2;
        there >>= first;
        auto up_to = [](int keys) {   // the lane's keys below `keys`, counted from its first
            return (1u << min(max(keys, 0), 4)) - 1u | ((1u << min(max(keys - 16, 0), 4)) - 1u) << 16;
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            __builtin_amdgcn_sched_barrier(0);
            const int last = pos[n] - key0 - first;
            uint32_t mask = there & up_to(last + 1);
            if (a.window)
                mask &= ~up_to(last - a.window + 1);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[n][j >> 2][j & 3] = mask >> ((j >> 2) * 16 + (j & 3)) & 1 ? s[n][j >> 2][j & 3] : -INFINITY;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // The weights of 32 keys, and what they do to the maximum and the sum. The maximum follows only when a score
    // exceeds it by kLag: until then weights are larger than one, which costs no bits, and o stays as it is.
    // One fused operation scales a score and takes the maximum's product from it. That product's rounding is in all exponents
    // made under one maximum, but those of other waves, of other parts and of the keys before the maximum moved have another,
    // and the joins know of neither: weights of two maxima are off against each other by up to 2^-23 of the product, times
    // ln 2. Up to kFused that is 2^-10 (bf16) or 2^-13 (fp16), a quarter of the weights' own rounding. Under larger maxima, and for fp32
    // rows, for which all weights would have to be that much more exact, scores are subtracted first. (With a limit of 2^20, sums
    // of two maxima near scores of 7e5 were off by 4%.)
    static constexpr float kFused = std::is_same<T, F16>::value ? 0x1p10f : 0x1p13f;
    __device__ __forceinline__ void weigh(const AttnArgs &a, const v4f (&s)[NT][2], uint4 (&p)[NT][kParts])
    {
        float top[NT];
        bool more = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            top[n] = fmaxf(fmaxf(larger(s[n][0][0], s[n][0][1]), larger(s[n][0][2], s[n][0][3])),
                           fmaxf(larger(s[n][1][0], s[n][1][1]), larger(s[n][1][2], s[n][1][3])));
            more |= (top[n] - m[n]) * c(a, n) > kLag;
        }
        if (rarely(__any(more))) {
            bool fine = true;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
                top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
                const float now = fmaxf(m[n], top[n]);
                const float f = now > m[n] ? __builtin_amdgcn_exp2f((m[n] - now) * c(a, n)) : 1.0f;
                m[n] = now;
                fine &= fabsf(now) * c(a, n) < kFused || now == -INFINITY;
                l[n] *= f;
#pragma unroll
                for (int d = 0; d < kO; ++d)
                    o[n][d] *= f;
            }
            small = __all(fine);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            __builtin_amdgcn_sched_barrier(0);   // a tile's weights at a time
            const float base = m[n] == -INFINITY ? 0.0f : m[n];   // no key yet: all weights are 0
            float w[8];
            if (!EXACT && !rarely(!small)) {
                const float neg = __builtin_fmaf(-base, c(a, n), kBias);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = __builtin_fmaf(s[n][j >> 2][j & 3], c(a, n), neg);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = EXACT ? (s[n][j >> 2][j & 3] - base) * c(a, n) : __builtin_fmaf(s[n][j >> 2][j & 3] - base, c(a, n), kBias);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = __builtin_amdgcn_exp2f(w[j]) * (EXACT ? kUnit : 1.0f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t parts[kParts];
                Split<T, EXACT>::pair(w[2 * x], w[2 * x + 1], parts);
#pragma unroll
                for (int y = 0; y < kParts; ++y)
                    word(p[n][y], x) = parts[y];
                if constexpr (EXACT)
                    l[n] += w[2 * x] + w[2 * x + 1];
                else
                    l[n] = dot2(parts[0], ones(T()), l[n], T());   // the weights as they are used
            }
        }
    }
    struct Values {
        uint4 v[AHEAD ? kO : 1];
    };
    __device__ __forceinline__ void read_ahead(const lds_t *vb, Values &w) const
    {
        if constexpr (AHEAD) {
#pragma unroll
            for (int d = 0; d < kO; ++d)
                w.v[d] = value(vb, d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __device__ __forceinline__ void add(const lds_t *vb, const Values &w, const uint4 (&p)[NT][kParts])
    {
        if constexpr (AHEAD) {
#pragma unroll
            for (int y = kParts; y-- > 0;)
#pragma unroll
                for (int d = 0; d < kO; ++d)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        o[n][d] = mfma(w.v[d], p[n][y], o[n][d], T());
        } else {
            constexpr int kBatch = NT > 1 ? 2 : 4, kBatches = kO / kBatch;
            uint4 v[2][kBatch];
            auto read = [&](int b) {
#pragma unroll
                for (int x = 0; x < kBatch; ++x)
                    v[b & 1][x] = value(vb, b * kBatch + x);
            };
            read(0);
#pragma unroll
            for (int b = 0; b < kBatches; ++b) {
                if (b + 1 < kBatches)
                    read(b + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int y = kParts; y-- > 0;)
#pragma unroll
                    for (int x = 0; x < kBatch; ++x)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            o[n][b * kBatch + x] = mfma(v[b & 1][x], p[n][y], o[n][b * kBatch + x], T());
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // The elements of key k's values (in memory at v) that are not finite, into the rows that see it: LDS holds zeros in their
    // place, as a weight of 0 would not keep them from the other rows.
    __device__ __forceinline__ void poison(const AttnArgs &a, int k, const uint8_t *v, int lane)
    {
        v = uniform(v);
        uint32_t off = 8 * (lane >> 4);
#pragma unroll
        for (int d = 0; d < kO; ++d) {
            asm volatile("" : "+v"(off)::"memory");   // one load at a time, see hide()
            __builtin_amdgcn_sched_barrier(0);
            const uint2 two = __builtin_bit_cast(uint2, *(const __attribute__((address_space(1))) v2u *)(v + 32 * d + off));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                unpack(i < 2 ? two.x : two.y, lo, hi, T());
                const float e = i & 1 ? hi : lo, odd = fabsf(e) < INFINITY ? 0.0f : e;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    o[n][d][i] += sees(a, n, k) ? odd : 0.0f;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // the rows' sums, in all four lanes that share one
    __device__ __forceinline__ void end()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
        }
    }
};

// Zeros in LDS for the values of keys that no row of the unit sees (memory that no one has written, or another
// request's), and for those that are not finite: a weight of 0 would not keep either from a row that does not see the key.
// KEYS keys of D elements from `buf` on, bit x of `there` set if key x is seen; taken by LANES threads of which
// this is number `me`. Returns the keys that are seen and have such values (see Rows::poison), as far as this thread has met them.
template <int D, class T, int LANES, int KEYS>
__device__ __forceinline__ uint64_t clean(lds_t *buf, uint64_t there, int me)
{
    constexpr int kLanes = D / 8, kPasses = KEYS * kLanes / LANES;   // threads of a row
    static_assert(LANES % kLanes == 0 && kPasses >= 1, "whole rows");
    uint64_t strange = 0;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
        const int x = pass * (LANES / kLanes) + me / kLanes;
        __attribute__((address_space(3))) v4u *at = (__attribute__((address_space(3))) v4u *)(buf + (x >> 4) * Lay<D>::kGroup + Lay<D>::row(x & 15) + me % kLanes * 16);
        v4u v = *at;
        const bool seen = there >> x & 1;
        bool odd = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            constexpr uint32_t e = exponents(T()), lo = e & 0xffffu, hi = e & 0xffff0000u;
            const uint32_t bad = ((v[w] & lo) == lo ? 0xffffu : 0u) | ((v[w] & hi) == hi ? 0xffff0000u : 0u);
            odd |= bad != 0;
            v[w] = seen ? v[w] & ~bad : 0u;
        }
        if (odd || !seen)
            *at = v;
        if (odd && seen)
            strange |= 1ull << x;
    }
    return strange;
}
// keys lo .. hi - 1 as bits of those from key0 on
__device__ __forceinline__ uint64_t key_bits(int lo, int hi, int key0)
{
    auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
    return below(hi - key0) & ~below(lo - key0);
}
__device__ __forceinline__ uint64_t any_of(uint64_t bits)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        bits |= (uint64_t)__shfl_xor((unsigned long long)bits, d);
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(bits >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)bits);
}

// ---- results ------------------------------------------------------------------------
// o[0..3] / l, gated, as elements d .. d + 3 of the unit's row `row`
template <class Q, int D>
__device__ __forceinline__ void put_out(const AttnArgs &a, int first, int group_row, int head, int d, v4f o, float l)
{
    const int tok = by_group(a, group_row), h = head * a.group + group_row - tok * a.group;
    const size_t t = (size_t)(first + tok);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = l == 0.0f ? 0.0f : o[i] / l;
    if (a.gate) {
        const size_t at = (size_t)((long long)t * a.g_row + (long long)h * a.g_head) + d;
        float g[4];
        if (a.gate_dtype == TB_F32) {
            const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.gate) + at);
            g[0] = w.x, g[1] = w.y, g[2] = w.z, g[3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.gate) + at);
            if (a.gate_dtype == TB_BF16) {
                unpack(w.x, g[0], g[1], Bf16());
                unpack(w.y, g[2], g[3], Bf16());
            } else {
                unpack(w.x, g[0], g[1], F16());
                unpack(w.y, g[2], g[3], F16());
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = v[i] / (1.0f + expf(-g[i]));
    }
    const size_t at = (t * ((size_t)a.kv_heads * a.group) + h) * D + d;
    if constexpr (std::is_same<Q, float>::value)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = make_uint2(pack(v[0], v[1], Q()), pack(v[2], v[3], Q()));
}

// What the second launch needs to know of the unit that begins in a slot and ends in another
struct Meta {
    int parts, head, first, rows, row0, pad[3];
};

// Partial results of slot s: [0] of the unit that began before it, [1] of the one that begins in it.
// ROWS x D sums, then ROWS maxima, ROWS sums of weights and ROWS factors of the scores.
template <int ROWS, int D>
__device__ __forceinline__ float *part_of(const AttnArgs &a, int slot, bool begins)
{
    return a.part + ((size_t)slot * 2 + begins) * (ROWS * (D + 3));
}

// ---- few rows: a unit has 16 rows, its keys are split over the waves -----------------
// A wave takes every fourth block of 32 keys, through buffers of its own: no barriers, and a wave's next keys are
// on their way while it multiplies its values, and the other way round.
// Bound: memory, behind a chain of latencies. One fp32 token of 16 heads over 131072 keys of 2 x 256 bf16: the loops
// read 268 MB in 38 us, 7 TB/s (some of it from the last cache: memory alone gives 5.9); 9 us before them (the line of units 1.5, pages and q 2.8, the first keys) and 4 after; the
// join 8. The same over 4096 keys: 15 us, of which no part is over 2, and 7.
constexpr int kNarrowWaves = 4, kNarrowRows = 16, kNarrowStep = kNarrowWaves * kBlk;
constexpr int kNarrowExtra = 2;   // in steps: 48 ragged requests, 0: 71 us, 2: 47

// workgroups of a CU: what LDS holds (128, 64 or 32 KB each), and registers
constexpr int narrow_per_cu(int dim) { return dim == 256 ? 1 : dim == 128 ? 2 : 3; }

template <int D, class T, class Q>
__global__ __launch_bounds__(kNarrowWaves * 64, narrow_per_cu(D)) void attn_narrow_kernel(AttnArgs a)
{
    constexpr bool kExact = std::is_same<Q, float>::value;
    using R = Rows<D, T, kExact, 1, !kExact || D < 256>;
    constexpr int kGroup = Lay<D>::kGroup, kBuf = 2 * kGroup;
    // arrays of their own: a read of one then waits for no load of the other
    __shared__ __align__(128) uint8_t kbuf[kNarrowWaves * kBuf];
    __shared__ __align__(128) uint8_t vbuf[kNarrowWaves * kBuf];
    __shared__ int chunk_s[kNarrowWaves * 64];
    __shared__ int wave_s[kNarrowWaves], found_s[6];
    __shared__ float m_s[kNarrowWaves][kNarrowRows], l_s[kNarrowWaves][kNarrowRows], c_s[kNarrowRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
    // neighbours on the line of units share keys: they go to the same XCD (workgroup b runs on XCD b % 8)
    const int slots = gridDim.x, slot = (int)(blockIdx.x & 7) * (slots >> 3) + (int)(blockIdx.x >> 3);
    Start st;
    unsigned per;
    find_start<kNarrowRows, kNarrowStep, kNarrowExtra, kNarrowWaves>(a, slots, slot, chunk_s, wave_s, found_s, st, per);
    unsigned line = (unsigned)slot * per;
    const unsigned end = min(line + per, (unsigned)st.all * (unsigned)a.kv_heads);
    Meta *meta = reinterpret_cast<Meta *>(a.meta) + slot;
    int parts = 0;
    if (line < end) {
        lds_t *kb = (lds_t *)kbuf + wave * kBuf, *vb = (lds_t *)vbuf + wave * kBuf;
        const const_ints table = (const_ints)a.table;
        int head = (int)(line / (unsigned)st.all), req = st.req, into = st.into;
        Unit u = st.u;
        Loader<D> loader;
        loader.init(lane);
        R rows;
        rows.init_reads(lane);
        for (;;) {
            span<kNarrowRows, kNarrowStep, kNarrowExtra>(a, u);
            // [into, into + here) of the unit's place on the line: steps from .. to, if any
            const int here = (int)min((unsigned)(u.cost - into), end - line);
            const int from = max(into - kNarrowExtra, 0), take = into + here - kNarrowExtra - from;
            if (take > 0) {
                const int row0 = u.tile * kNarrowRows, nrows = min(u.n * a.group - row0, kNarrowRows);

                // all rows see keys from some_lo on up to some_hi; any row, those from kbeg on up to kend
                int some_lo = 0, some_hi;
                {
                    const int p0 = u.len - u.n + by_group(a, row0), p1 = u.len - u.n + by_group(a, row0 + nrows - 1);
                    some_hi = max(min(u.kend, p0 + 1), 0);
                    if (a.window)
                        some_lo = max(p1 - a.window + 1, 0);
                }
                const int hi = min((u.s0 + from + take) * kNarrowStep, u.kend);
                int blk = (u.s0 + from) * kNarrowWaves + wave;
                while ((blk + 1) * kBlk <= u.kbeg)
                    blk += kNarrowWaves;
                // The pages of a block's two groups of 16 keys, read a block ahead; then the groups' places. A group without a page
                // is read from page 0, and not used.
                auto ids_of = [&](int b, int (&id)[2]) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        id[t] = table[(size_t)req * a.width + (min(b * kBlk + 16 * t, u.kend - 1) >> a.page_shift)];
                };
                auto place = [&](int b, const int (&id)[2], size_t (&at)[2]) {
                    uint32_t gone = 0;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int key = b * kBlk + 16 * t;
                        const bool page = (unsigned)id[t] < (unsigned)a.pages;
                        gone |= page && key < u.kend ? 0u : 1u << t;
                        at[t] = ((((size_t)(page ? id[t] : 0) * a.kv_heads + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * (D * 2);
                    }
                    return gone;
                };
                int id[2] = {-1, -1};
                const bool any = blk * kBlk < hi;
                if (any)
                    ids_of(blk, id);
                typename R::Raw raw;
                rows.fetch(a, u, head, row0, opaque(lane), raw);
                rows.begin(a, raw);
                size_t at[2] = {0, 0};
                uint32_t gone = 0;
                if (any) {
                    gone = place(blk, id, at);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        loader.load(a.k + at[t], kb + t * kGroup);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        loader.load(a.v + at[t], vb + t * kGroup);
                    ids_of(blk + kNarrowWaves, id);
                }
                while (blk * kBlk < hi) {
                    const int key0 = blk * kBlk, next = blk + kNarrowWaves;
                    const bool more = next * kBlk < hi;
                    size_t nat[2] = {0, 0};
                    uint32_t ngone = 0;
                    v4f s[1][2];
                    landed<2 * Loader<D>::kLoads>();   // all but the values, which were asked for last
                    rows.scores(kb, s);
                    lds_read();
                    if (more) {
                        ngone = place(next, id, nat);
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            loader.load(a.k + nat[t], kb + t * kGroup);
                    }
                    const bool whole = key0 >= some_lo && key0 + kBlk <= some_hi && !gone;
                    const uint32_t there = (uint32_t)key_bits(u.kbeg, u.kend, key0) & ~((gone & 1 ? 0xffffu : 0u) | (gone & 2 ? 0xffff0000u : 0u));
                    if (rarely(!whole))
                        rows.hide(a, key0, lane, there, s);
                    if (more)   // the next keys may be on their way
                        landed<2 * Loader<D>::kLoads>();
                    else
                        landed<0>();
                    uint64_t strange = 0;
                    if (rarely(!whole)) {
                        strange = any_of(clean<D, T, 64, kBlk>(vb, there, lane));
                        lds_read();
                    }
                    typename R::Values values;
                    rows.read_ahead(vb, values);
                    uint4 p[1][R::kParts];
                    rows.weigh(a, s, p);
                    if (rarely(strange != 0))
                        for (; strange; strange &= strange - 1) {
                            const int x = __builtin_ctzll(strange), t = x >> 4;
                            rows.poison(a, key0 + x, a.v + (t ? at[1] : at[0]) + (x & 15) * (D * 2), lane);
                        }
                    rows.add(vb, values, p);
                    lds_read();
                    if (more) {
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            loader.load(a.v + nat[t], vb + t * kGroup);
                        ids_of(next + kNarrowWaves, id);
                    }
                    gone = ngone;
                    at[0] = nat[0], at[1] = nat[1];
                    blk = next;
                }
                rows.end();

                // the waves' sums become one, in the order of the waves
                if (g == 0) {
                    m_s[wave][i] = rows.m[0];
                    l_s[wave][i] = rows.l[0];
                    c_s[i] = rows.c(a, 0);   // the same in all waves
                }
                __syncthreads();
                float top = m_s[0][i];
#pragma unroll
                for (int w = 1; w < kNarrowWaves; ++w)
                    top = fmaxf(top, m_s[w][i]);
                const float f = rows.m[0] == top ? 1.0f : __builtin_amdgcn_exp2f((rows.m[0] - top) * rows.c(a, 0));
                float *mine = reinterpret_cast<float *>(kbuf + wave * kBuf);
#pragma unroll
                for (int d = 0; d < R::kO; ++d)
                    *reinterpret_cast<v4f *>(mine + i * D + ((4 * d + g) ^ i) * 4) = rows.o[0][d] * f;
                __syncthreads();
                const bool begins = from == 0, ends = from + take == u.steps;
                for (int x = tid; x < kNarrowRows * D / 4; x += kNarrowWaves * 64) {
                    const int r = x / (D / 4), ch = x % (D / 4);
                    float best = m_s[0][r];
#pragma unroll
                    for (int w = 1; w < kNarrowWaves; ++w)
                        best = fmaxf(best, m_s[w][r]);
                    v4f o = {};
                    float l = 0.0f;
#pragma unroll
                    for (int w = 0; w < kNarrowWaves; ++w) {
                        o += *reinterpret_cast<const v4f *>(reinterpret_cast<const float *>(kbuf + w * kBuf) + r * D + (ch ^ r) * 4);
                        const float mw = m_s[w][r];
                        l += l_s[w][r] * (mw == best ? 1.0f : __builtin_amdgcn_exp2f((mw - best) * c_s[r]));
                    }
                    if (begins && ends) {
                        if (r < nrows)
                            put_out<Q, D>(a, u.first, row0 + r, head, ch * 4, o, l);
                    } else {
                        float *part = part_of<kNarrowRows, D>(a, slot, begins);
                        *reinterpret_cast<v4f *>(part + r * D + ch * 4) = o;
                        if (ch == 0) {
                            part[kNarrowRows * D + r] = best;
                            part[kNarrowRows * D + kNarrowRows + r] = l;
                            part[kNarrowRows * D + 2 * kNarrowRows + r] = c_s[r];
                        }
                    }
                }
                if (begins && !ends) {
                    // the unit's last place on the line is line - into + cost - 1
                    parts = (int)((line - (unsigned)into + (unsigned)u.cost - 1u) / per) - slot + 1;
                    if (tid == 0)
                        *meta = Meta{parts, head, u.first, u.n * a.group, row0, {}};
                }
            }
            line += here;
            if (line >= end)
                break;
            // the next unit
            into = 0;
            ++u.tile;
            if (u.tile * kNarrowRows >= u.n * a.group) {
                u.tile = 0;
                do {
                    if (++req == a.requests) {
                        req = 0;
                        ++head;
                    }
                    int f, n, len;
                    request_of(a, req, f, n, len);
                    u.first = __builtin_amdgcn_readfirstlane(f);
                    u.n = __builtin_amdgcn_readfirstlane(n);
                    u.len = __builtin_amdgcn_readfirstlane(len);
                } while (u.n == 0);   // line < end: there is one
            }
            __syncthreads();
        }
    }
    if (parts == 0 && tid == 0)
        meta->parts = 0;
}

// ---- many rows: a unit has a tile of rows for each wave, which all read the same keys ----------------
// wide_step keys and their values at a time, in buffers of which one is multiplied while the others are filled. Each operand
// that is read from LDS enters two instructions, for two tiles of 16 rows.
//   D = 256: o and q take 192 of 256 registers, and the loop has none to spare. Eight waves share the buffers: with four of
//   them in two workgroups a CU, the same number of cycles, but twice the loads, and a lower clock (357 us against 333).
//   D = 128: two workgroups a CU, 32 keys a step and four buffers (a mixed step of 12 requests: 73 us; 64 keys and two
//   buffers 75; eight waves that share 64 keys 77; three workgroups a CU the same as two).
// Bound: the loop's waits. 2048 new bf16 tokens behind 8192, 16 heads of 256: 301 to 325 us with the join, 0.95 to 1.03
// PFLOP/s; under counters, at 1.9 GHz, the matrix cores are busy in 47% of the cycles, and vector operations take another 30%. A
// library product of 8192^3 reaches 1.19 to 1.26. Rows in fp32, three products for one: 680 to 716. 16 heads on 4 x 64: 132.
// wide_extra: what beginning and ending a unit takes, in steps. D = 256: q and the first keys 6 us, rows out 4 to 11; D = 128, 12
// requests with chunks of up to 509: 3 and 5, beside 1.5 a step.
constexpr int wide_extra(int dim) { return dim == 256 ? 6 : 8; }
constexpr int wide_step(int dim) { return dim == 256 ? 64 : 32; }     // keys
constexpr int wide_buffers(int dim) { return dim == 256 ? 2 : 4; }
constexpr int wide_waves(int dim) { return dim == 256 ? 8 : 4; }
constexpr int wide_tiles(bool exact) { return exact ? 1 : 2; }
constexpr int wide_rows(int dim, bool exact) { return wide_waves(dim) * wide_tiles(exact) * 16; }
constexpr int wide_per_cu(int dim) { return dim == 256 ? 1 : dim == 128 ? 2 : 4; }   // workgroups

template <int D, class T, class Q>
__global__ __launch_bounds__(wide_waves(D) * 64, wide_waves(D) / 4 * wide_per_cu(D)) void attn_wide_kernel(AttnArgs a)
{
    constexpr bool kExact = std::is_same<Q, float>::value;
    constexpr int kWaves = wide_waves(D), kTiles = wide_tiles(kExact), kRows = wide_rows(D, kExact);
    constexpr int kStep = wide_step(D), kBufs = wide_buffers(D), kExtra = wide_extra(D);
    using R = Rows<D, T, kExact, kTiles, D < 256>;
    constexpr int kGroup = Lay<D>::kGroup, kGroups = kStep / 16, kBuf = kGroups * kGroup;
    __shared__ __align__(128) uint8_t kbuf[kBufs * kBuf];
    __shared__ __align__(128) uint8_t vbuf[kBufs * kBuf];
    __shared__ int chunk_s[kWaves * 64];
    __shared__ int wave_s[kWaves], found_s[6];
    __shared__ unsigned long long strange_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slots = gridDim.x, slot = (int)(blockIdx.x & 7) * (slots >> 3) + (int)(blockIdx.x >> 3);
    if (tid == 0)
        strange_s = 0;
    Start st;
    unsigned per;
    find_start<kRows, kStep, kExtra, kWaves>(a, slots, slot, chunk_s, wave_s, found_s, st, per);
    unsigned line = (unsigned)slot * per;
    const unsigned end = min(line + per, (unsigned)st.all * (unsigned)a.kv_heads);
    Meta *meta = reinterpret_cast<Meta *>(a.meta) + slot;
    int parts = 0;
    if (line < end) {
        const const_ints table = (const_ints)a.table;
        int head = (int)(line / (unsigned)st.all), req = st.req, into = st.into;
        Unit u = st.u;
        Loader<D> loader;
        loader.init(lane);
        R rows;
        rows.init_reads(lane);
        for (;;) {
            span<kRows, kStep, kExtra>(a, u);
            // [into, into + here) of the unit's place on the line: steps from .. to, if any
            const int here = (int)min((unsigned)(u.cost - into), end - line);
            const int from = max(into - kExtra, 0), take = into + here - kExtra - from;
            if (take > 0) {
                const int unit0 = u.tile * kRows, nrows = min(u.n * a.group - unit0, kRows);
                const int row0 = unit0 + wave * kTiles * 16;
                const bool active = row0 < unit0 + nrows;   // the wave has rows
                // The wave's rows all see the keys from some_lo on up to some_hi; any of them, those from any_lo on up to any_hi.
                int some_lo = 0, some_hi = 0, any_lo = 0, any_hi = 0;
                if (active) {
                    const int last = min(row0 + kTiles * 16, unit0 + nrows) - 1;
                    const int p0 = u.len - u.n + by_group(a, row0), p1 = u.len - u.n + by_group(a, last);
                    some_hi = max(min(u.kend, p0 + 1), 0);
                    any_hi = max(min(u.kend, p1 + 1), 0);
                    if (a.window) {
                        some_lo = max(p1 - a.window + 1, 0);
                        any_lo = max(p0 - a.window + 1, 0);
                    }
                }
                const int first = u.s0 + from;
                // all rows of the unit see the keys from unit_lo on up to unit_hi
                const int unit_hi = min(u.kend, u.len - u.n + by_group(a, unit0) + 1);
                const int unit_lo = a.window ? u.len - u.n + by_group(a, unit0 + nrows - 1) - a.window + 1 : 0;
                // Of a step: group x of 16 keys; its page, if it has one; and the place of a key in the cache's arrays
                auto id_of = [&](int key) { return table[(size_t)req * a.width + (min(key, max(u.kend - 1, 0)) >> a.page_shift)]; };
                auto at_of = [&](int id, int key) {
                    id = (unsigned)id < (unsigned)a.pages ? id : 0;
                    return ((((size_t)id * a.kv_heads + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * (D * 2);
                };
                // The groups' keys and values are loaded by the waves in turn: items 2 x and 2 x + 1 are those of group x. A
                // wave's pages are read a step ahead.
                constexpr int kItems = 2 * kGroups / kWaves;
                static_assert(kItems * kWaves == 2 * kGroups && kItems <= 2, "one item for each wave, or the keys and the values of a group");
                const int mine16 = (wave * kItems >> 1) * 16;
                auto load = [&](int step, int b, int id) {
                    const size_t at = at_of(id, step * kStep + mine16);
                    const int to = b * kBuf + (wave * kItems >> 1) * kGroup;
                    if (kItems == 2 || !(wave & 1))
                        loader.load(a.k + at, (lds_t *)kbuf + to);
                    if (kItems == 2 || (wave & 1))
                        loader.load(a.v + at, (lds_t *)vbuf + to);
                };
                // The pages of a step's groups, read a step ahead; from them, the keys that some row sees
                constexpr uint64_t kAll = kStep == 64 ? ~0ull : (1ull << kStep % 64) - 1;
                int ids[kGroups];
                auto read_ids = [&](int step) {
#pragma unroll
                    for (int x = 0; x < kGroups; ++x)
                        ids[x] = id_of(step * kStep + 16 * x);
                };
                auto there_of = [&](int step) {
                    uint64_t there = kAll;
                    if (step * kStep < u.kbeg || (step + 1) * kStep > u.kend)
                        there &= key_bits(u.kbeg, u.kend, step * kStep);
#pragma unroll
                    for (int x = 0; x < kGroups; ++x)
                        if ((unsigned)ids[x] >= (unsigned)a.pages)
                            there &= ~(0xffffull << (16 * x));
                    return there;
                };
                // the first steps' loads; the wave's page of the step after them; the first step's keys
                int next_id = id_of(first * kStep + mine16);
                typename R::Raw raw;
                rows.fetch(a, u, head, row0, opaque(lane), raw);
#pragma unroll
                for (int x = 0; x < kBufs - 1; ++x) {
                    if (x < take)
                        load(first + x, x, next_id);
                    next_id = id_of((first + x + 1) * kStep + mine16);
                }
                read_ids(first);
                rows.begin(a, raw);
                for (int x = 0; x < take; ++x) {
                    const int b = x % kBufs, step = first + x, step0 = step * kStep;
                    // this step's loads have landed: of the wave's own by the wait, of the others' by the barrier; and what
                    // was read in the step before may be overwritten
                    if (take - 1 - x >= kBufs - 2)
                        landed<kItems * Loader<D>::kLoads * (kBufs - 2)>();
                    else
                        landed<0>();
                    __syncthreads();
                    const uint64_t there = there_of(step);
                    read_ids(step + 1);
                    uint64_t strange = 0;
                    if (rarely(step0 < unit_lo || step0 + kStep > unit_hi || there != kAll)) {
                        const uint64_t odd = any_of(clean<D, T, kWaves * 64, kStep>((lds_t *)vbuf + b * kBuf, there, opaque(tid)));
                        if (odd && lane == 0)
                            atomicOr(&strange_s, (unsigned long long)odd);
                        __syncthreads();
                        strange = any_of(strange_s);
                    }
                    if (x + kBufs - 1 < take) {
                        loader.pin();
                        load(step + kBufs - 1, (x + kBufs - 1) % kBufs, next_id);
                        next_id = id_of((step + kBufs) * kStep + mine16);
                    }
#pragma unroll 1
                    for (int y = 0; y < kStep / kBlk; ++y) {
                        const int key0 = step0 + y * kBlk;
                        if (key0 >= any_hi || key0 + kBlk <= any_lo)
                            continue;
                        const lds_t *kb = (const lds_t *)kbuf + b * kBuf + y * 2 * kGroup, *vb = (const lds_t *)vbuf + b * kBuf + y * 2 * kGroup;
                        const uint32_t mine = (uint32_t)(there >> (32 * y));
                        v4f s[kTiles][2];
                        rows.scores(kb, s);
                        if (rarely(key0 < some_lo || key0 + kBlk > some_hi || ~mine))
                            rows.hide(a, key0, opaque(lane), mine, s);
                        typename R::Values values;
                        rows.read_ahead(vb, values);
                        uint4 p[kTiles][R::kParts];
                        rows.weigh(a, s, p);
                        if (rarely((uint32_t)(strange >> (32 * y)) != 0))
                            for (uint32_t odd = (uint32_t)(strange >> (32 * y)); odd; odd &= odd - 1) {
                                const int key = key0 + __builtin_ctz(odd);
                                rows.poison(a, key, a.v + at_of(id_of(key), key), opaque(lane));
                            }
                        rows.add(vb, values, p);
                    }
                    if (strange) {
                        __syncthreads();   // all have read it
                        if (tid == 0)
                            strange_s = 0;
                    }
                }
                __syncthreads();
                rows.end();
                const bool begins = from == 0, ends = from + take == u.steps;
                // Through LDS, a column tile at a time, so that whole rows are written. (Both buffers have been read; a wave
                // reads what its own lanes wrote.)
                float *mine = reinterpret_cast<float *>(wave < kWaves / 2 ? kbuf : vbuf) + wave % (kWaves / 2) * (16 * D);
                const int own = opaque(lane), i = own & 15, g = own >> 4;
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    const int r0 = wave * kTiles * 16 + 16 * n;   // of the unit
#pragma unroll
                    for (int d = 0; d < R::kO; ++d)
                        *reinterpret_cast<v4f *>(mine + i * D + ((4 * d + g) ^ i) * 4) = rows.o[n][d];
                    lds_read();
                    const float ln = rows.l[n], mn = rows.m[n], cn = rows.c(a, n);
#pragma unroll 1
                    for (int x = own; x < 4 * D; x += 64) {
                        const int r = x / (D / 4), ch = x % (D / 4);
                        const v4f o = *reinterpret_cast<const v4f *>(mine + r * D + (ch ^ r) * 4);
                        const float l = __shfl(ln, r), m = __shfl(mn, r), c = __shfl(cn, r);
                        if (r0 + r >= nrows)
                            continue;
                        if (begins && ends) {
                            put_out<Q, D>(a, u.first, unit0 + r0 + r, head, ch * 4, o, l);
                        } else {
                            float *part = part_of<kRows, D>(a, slot, begins);
                            *reinterpret_cast<v4f *>(part + (r0 + r) * D + ch * 4) = o;
                            if (ch == 0) {
                                part[kRows * D + r0 + r] = m;
                                part[kRows * D + kRows + r0 + r] = l;
                                part[kRows * D + 2 * kRows + r0 + r] = c;
                            }
                        }
                    }
                    lds_read();
                }
                __syncthreads();
                if (begins && !ends) {
                    parts = (int)((line - (unsigned)into + (unsigned)u.cost - 1u) / per) - slot + 1;
                    if (tid == 0)
                        *meta = Meta{parts, head, u.first, u.n * a.group, unit0, {}};
                }
            }
            line += here;
            if (line >= end)
                break;
            into = 0;
            ++u.tile;
            if (u.tile * kRows >= u.n * a.group) {
                u.tile = 0;
                do {
                    if (++req == a.requests) {
                        req = 0;
                        ++head;
                    }
                    int f, n, len;
                    request_of(a, req, f, n, len);
                    u.first = __builtin_amdgcn_readfirstlane(f);
                    u.n = __builtin_amdgcn_readfirstlane(n);
                    u.len = __builtin_amdgcn_readfirstlane(len);
                } while (u.n == 0);   // line < end: there is one
            }
        }
    }
    if (parts == 0 && tid == 0)
        meta->parts = 0;
}

// ---- units that a border cut ---------------------------------------------------------
// o = sum_j 2^(c (m_j - m)) o_j and l likewise, over the parts in order, for the units that begin in a slot and end in
// another.
// Few rows, many parts: workgroup (slot, y) takes every so many rows from row y on. Its threads are as many groups as hold a row at a time, and
// a group takes every so many parts; their sums are added in the order of the groups.
template <int D, class Q, int THREADS>
__global__ __launch_bounds__(THREADS) void attn_join_narrow_kernel(AttnArgs a)
{
    constexpr int kLanes = D / 4, kGroups = THREADS / kLanes, kWaves = THREADS / 64, kMost = 768;
    static_assert(narrow_per_cu(D) * 256 <= kMost, "as many parts as slots at most");
    __shared__ float weight_s[kMost];
    __shared__ v4f sum_s[THREADS];
    __shared__ float wave_s[2][kWaves];
    const int slot = blockIdx.x, tid = threadIdx.x, group = tid / kLanes, d = tid % kLanes * 4;
    const Meta meta = reinterpret_cast<const Meta *>(a.meta)[slot];
    if (meta.parts == 0)
        return;
    for (int r = blockIdx.y; r < kNarrowRows && meta.row0 + r < meta.rows; r += gridDim.y) {
        // part j, 0 of which is the slot's own
        auto part = [&](int j) { return part_of<kNarrowRows, D>(a, slot + j, j == 0); };
        constexpr int kM = kNarrowRows * D, kL = kM + kNarrowRows, kC = kL + kNarrowRows;
        const float c = part(0)[kC + r];
        float best = -INFINITY;
        for (int j = tid; j < meta.parts; j += THREADS) {
            weight_s[j] = part(j)[kM + r];
            best = fmaxf(best, weight_s[j]);
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1)
            best = fmaxf(best, __shfl_xor(best, x));
        if ((tid & 63) == 0)
            wave_s[0][tid >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kWaves; ++x)
            best = fmaxf(best, wave_s[0][x]);
        float l = 0.0f;
        for (int j = tid; j < meta.parts; j += THREADS) {
            const float m = weight_s[j], f = m == best ? 1.0f : __builtin_amdgcn_exp2f((m - best) * c);
            weight_s[j] = f;
            l += part(j)[kL + r] * f;
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1)
            l += __shfl_xor(l, x);
        if ((tid & 63) == 0)
            wave_s[1][tid >> 6] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int x = 0; x < kWaves; ++x)
            l += wave_s[1][x];
        v4f o = {};
        constexpr int kAhead = 8;   // parts of a group whose loads are in flight
        for (int j0 = group; j0 < meta.parts; j0 += kAhead * kGroups) {
            v4f x[kAhead];
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const int j = min(j0 + y * kGroups, meta.parts - 1);
                x[y] = *reinterpret_cast<const v4f *>(part(j) + r * D + d);
            }
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const int j = j0 + y * kGroups;
                if (j < meta.parts)
                    o += x[y] * weight_s[j];
            }
        }
        sum_s[tid] = o;
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int x = 1; x < kGroups; ++x)
                o += sum_s[x * kLanes + tid];
            put_out<Q, D>(a, meta.first, meta.row0 + r, meta.head, d, o, l);
        }
        __syncthreads();   // the next row's weights and sums take this one's place
    }
}

// Many rows, few parts: workgroup (slot, y) takes 4 KB of the unit's rows, four parts at a time.
template <int ROWS, int D, class Q>
__global__ __launch_bounds__(256) void attn_join_wide_kernel(AttnArgs a)
{
    constexpr int kRows = 1024 / D, kLanes = D / 4, kAhead = 4;   // rows of the workgroup, threads of a row
    const int slot = blockIdx.x, d = threadIdx.x % kLanes * 4, r = blockIdx.y * kRows + threadIdx.x / kLanes;
    const Meta meta = reinterpret_cast<const Meta *>(a.meta)[slot];
    if (meta.parts == 0 || r >= ROWS || meta.row0 + r >= meta.rows)
        return;
    auto part = [&](int j) { return part_of<ROWS, D>(a, slot + j, j == 0); };
    constexpr int kM = ROWS * D, kL = kM + ROWS, kC = kL + ROWS;
    const float c = part(0)[kC + r];
    float best = -INFINITY, l = 0.0f;
    v4f o = {};
    for (int j0 = 0; j0 < meta.parts; j0 += kAhead) {
        v4f x[kAhead];
        float m[kAhead], s[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const float *p = part(min(j0 + y, meta.parts - 1));
            x[y] = *reinterpret_cast<const v4f *>(p + r * D + d);
            m[y] = p[kM + r];
            s[y] = p[kL + r];
        }
        float now = best;
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
            now = fmaxf(now, m[y]);
        const float f = best == now ? 1.0f : __builtin_amdgcn_exp2f((best - now) * c);
        o *= f;
        l *= f;
        best = now;
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            if (j0 + y < meta.parts) {
                const float g = m[y] == now ? 1.0f : __builtin_amdgcn_exp2f((m[y] - now) * c);
                o += x[y] * g;
                l += s[y] * g;
            }
        }
    }
    put_out<Q, D>(a, meta.first, meta.row0 + r, meta.head, d, o, l);
}

// ---- host ---------------------------------------------------------------------------
// Which kernel. The host knows no request's rows, only their sum. Times below are us with the kernel for few rows / for many, bf16.
//   More tokens than requests: one of them has several; it has (tokens - requests + 1) * group rows if the others bring one
//   each, and from 128 on the kernel for many rows runs. Beside a chunk it takes 0 to 40% longer for decodes, but the other one
//   walks all keys again for every 16 rows of the chunk. 16 heads on 2 x 256: 250 decodes of up to 8192 and 1000 tokens 527 / 337; 48
//   and 500 172 / 107; 12 and 64 behind 1000 33 / 46; 1 x 8 tokens behind 8192 34 / 54; 8 x 4 66 / 48; 64 x 4 210 / 213; 64 x 16
//   770 / 243. 24 heads on 8 x 128: 250 decodes and 1000 tokens 444 / 379; 64 x 4 behind 4096 192 / 205.
//   Else, as in decoding, a request has a token's heads. With more than 16 on a kv head, and many requests, they share their keys:
//   32 heads on 1 x 128 of 4 requests 30 / 66, of 32 42 / 31, of 128 55 / 45; 64 on 1 x 256 of 4 32 / 58, of 128 154 / 77.
//   (Requests that wait count here: 2048 tokens of one among 2048 are taken for decodes, 844 / 524.)
bool is_wide(int group, int requests, int tokens)
{
    const long long rows = (long long)tokens * group;
    return tokens > requests ? rows - (long long)(requests - 1) * group > 128 : group > 16 && rows >= 1024;
}

// As many workgroups as the chip's 256 CUs hold at a time: a constant, as the order of the sums must not depend
// on a partition's size.
int slots_of(bool wide, int dim) { return 256 * (wide ? wide_per_cu(dim) : narrow_per_cu(dim)); }
constexpr size_t kMetaBytes = 1024 * sizeof(Meta);   // as many as slots at most

size_t workspace(bool wide, int dim, bool exact)
{
    const int rows = wide ? wide_rows(dim, exact) : kNarrowRows;
    return kMetaBytes + (size_t)slots_of(wide, dim) * 2 * rows * (dim + 3) * 4;
}

template <int D, class T, class Q>
int launch(const AttnArgs &a, hipStream_t st)
{
    constexpr bool kExact = std::is_same<Q, float>::value;
    const bool wide = is_wide(a.group, a.requests, a.tokens);
    const int slots = slots_of(wide, D);
    if (wide)
        hipLaunchKernelGGL((attn_wide_kernel<D, T, Q>), dim3(slots), dim3(wide_waves(D) * 64), 0, st, a);
    else
        hipLaunchKernelGGL((attn_narrow_kernel<D, T, Q>), dim3(slots), dim3(kNarrowWaves * 64), 0, st, a);
    if (hipGetLastError() != hipSuccess)
        return TB_EHIP;
    constexpr int kRows = wide_rows(D, kExact);
    if (wide)
        hipLaunchKernelGGL((attn_join_wide_kernel<kRows, D, Q>), dim3(slots, kRows * D / 1024), dim3(256), 0, st, a);
    else {
        // Rows of a request while decoding, and threads for the parts of a unit: with a few of them, 1024 threads a row
        // cost more to start than they save (48 ragged requests: 9.9 us against 6; 1 of 131072: 8.1 against 15.6).
        const dim3 grid(slots, a.tokens <= a.requests ? std::min(a.group, kNarrowRows) : kNarrowRows);
        if ((long long)a.requests * a.kv_heads * 16 > slots)
            hipLaunchKernelGGL((attn_join_narrow_kernel<D, Q, 256>), grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((attn_join_narrow_kernel<D, Q, 1024>), grid, dim3(1024), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? TB_OK : TB_EHIP;
}

template <class T, class Q>
int launch_dim(int dim, const AttnArgs &a, hipStream_t st)
{
    return dim == 256 ? launch<256, T, Q>(a, st) : dim == 128 ? launch<128, T, Q>(a, st) : launch<64, T, Q>(a, st);
}

bool shapes_ok(const tb_kv_cache &c, int heads, int dtype, int requests, int tokens)
{
    return tbh::cache_ok(c) && heads >= 1 && heads % c.kv_heads == 0 && (dtype == TB_F32 || dtype == c.dtype) && requests >= 1 && tokens >= 1;
}
bool runs(const tb_kv_cache &c, int heads, int requests, int tokens)
{
    return (c.dim == 64 || c.dim == 128 || c.dim == 256) && requests <= 65536 && (long long)tokens * heads < (1ll << 30);
}

}  // namespace

// Enough for every call with at most these requests and tokens, whichever kernel it takes (see is_wide; a call wants its own kernel's)
extern "C" size_t tb_attn_paged_workspace_bytes(const tb_kv_cache *cache, int heads, int dtype, int requests, int tokens)
{
    if (!cache || !shapes_ok(*cache, heads, dtype, requests, tokens) || !runs(*cache, heads, requests, tokens))
        return 0;
    const int group = heads / cache->kv_heads;
    // one request with all the tokens; or one token of each of as many requests
    const bool wide = is_wide(group, 1, tokens) || is_wide(group, std::min(requests, tokens), std::min(requests, tokens));
    const size_t few = workspace(false, cache->dim, dtype == TB_F32);
    return wide ? std::max(few, workspace(true, cache->dim, dtype == TB_F32)) : few;
}

extern "C" int tb_attn_paged(const tb_heads *q, const tb_heads *gate, const tb_kv_cache *cache, const int32_t *table, int width,
                             const int32_t *offsets, const int32_t *lengths, int requests, int tokens, float scale, int window,
                             void *out, void *ws, size_t ws_bytes, void *stream)
{
    if (!q || !cache || !shapes_ok(*cache, q->heads, q->dtype, requests, tokens) || width < 1 || window < 0 || !(scale > 0.0f && scale * kLog2e < INFINITY))
        return TB_EINVAL;
    const int dim = cache->dim;
    if (gate && gate->heads != q->heads)
        return TB_EINVAL;
    const size_t qb = tbh::heads_bytes(*q, tokens, dim), gb = gate ? tbh::heads_bytes(*gate, tokens, dim) : 0;
    if (!qb || (gate && !gb))
        return TB_EINVAL;
    const bool can = runs(*cache, q->heads, requests, tokens);
    const size_t need = can ? workspace(is_wide(q->heads / cache->kv_heads, requests, tokens), dim, q->dtype == TB_F32) : 0;
    tbh::Arg a[9] = {{q->data, qb, false},
                     {cache->k, tbh::cache_bytes(*cache), false},
                     {cache->v, tbh::cache_bytes(*cache), false},
                     {table, (size_t)requests * (size_t)width * 4, false},
                     {offsets, (size_t)requests * 4 + 4, false},
                     {lengths, (size_t)requests * 4, false},
                     {out, (size_t)tokens * (size_t)q->heads * (size_t)dim * tbh::dtype_bytes(q->dtype), true},
                     {ws, ws_bytes, true}};
    size_t n = 8;
    if (gate)
        a[n++] = {gate->data, gb, false};
    if (int rc = tbh::check_args(a, n))
        return rc;
    const long long limit = (long long)width * cache->page;
    // the line of units, in steps of 32 keys at least and with what a unit costs beside them, is counted in 31 bits
    if (!can || limit > (1 << 30) ||
        ((long long)tokens * q->heads / 16 + (long long)requests * cache->kv_heads) * (limit / 32 + 10) >= (1ll << 31))
        return TB_EUNSUPPORTED;
    if (ws_bytes < need)
        return TB_EINVAL;
    AttnArgs r{};
    r.q = q->data, r.q_row = q->row_stride, r.q_head = q->head_stride;
    if (gate)
        r.gate = gate->data, r.g_row = gate->row_stride, r.g_head = gate->head_stride, r.gate_dtype = gate->dtype;
    r.k = static_cast<const uint8_t *>(cache->k), r.v = static_cast<const uint8_t *>(cache->v);
    r.table = table, r.offsets = offsets, r.lengths = lengths;
    r.pages = cache->pages, r.page_shift = tbh::log2_of(cache->page), r.width = width, r.kv_heads = cache->kv_heads;
    r.group = q->heads / cache->kv_heads;
    while ((1u << r.group_shift) < (uint32_t)r.group)
        ++r.group_shift;
    r.group_mul = (uint32_t)(((1ull << 32) * ((1ull << r.group_shift) - (uint64_t)r.group)) / (uint64_t)r.group + 1);
    r.requests = requests, r.tokens = tokens;
    r.window = std::min(window, 1 << 30), r.scale = scale * kLog2e, r.out = out;
    r.meta = static_cast<int32_t *>(ws), r.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kMetaBytes);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (cache->dtype == TB_BF16)
        return q->dtype == TB_F32 ? launch_dim<Bf16, float>(dim, r, st) : launch_dim<Bf16, Bf16>(dim, r, st);
    return q->dtype == TB_F32 ? launch_dim<F16, float>(dim, r, st) : launch_dim<F16, F16>(dim, r, st);
}
