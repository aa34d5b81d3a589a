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
// the rest is exact) or 22 (fp16: two). One part: rounded to nearest.
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
__device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// ---- units --------------------------------------------------------------------------
struct Unit {
    int first, n, len;   // the request's first row of q, its new tokens, its length
    int tile;
    int kbeg, kend;      // keys that any of its rows sees
    int s0, steps;       // its first step, in steps from key 0 on, and their number (one at least)
};

__device__ __forceinline__ void request_of(const AttnArgs &a, int r, int &first, int &n, int &len)
{
    first = min(max(a.offsets[r], 0), a.tokens);
    n = min(max(a.offsets[r + 1], first), a.tokens) - first;
    len = min(max(a.lengths[r], 0), 1 << 30);
}
template <int ROWS>
__device__ __forceinline__ int tiles_of(const AttnArgs &a, int n)
{
    return (n * a.group + ROWS - 1) / ROWS;
}
template <int ROWS, int STEP>
__device__ __forceinline__ void span(const AttnArgs &a, Unit &u)
{
    const int r0 = u.tile * ROWS, r1 = min(r0 + ROWS, u.n * a.group) - 1;
    const int p0 = u.len - u.n + r0 / a.group, p1 = u.len - u.n + r1 / a.group;
    u.kend = max(min(min(u.len, a.width << a.page_shift), p1 + 1), 0);
    u.kbeg = a.window ? min(max(p0 - a.window + 1, 0), u.kend) : 0;
    u.s0 = u.kbeg / STEP;
    u.steps = max((u.kend + STEP - 1) / STEP - u.s0, 1);
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
    int all;             // steps of all units of a kv head
    int req, tile, into; // the unit of the slot's first step, and its steps before that
};

// Every workgroup lays the whole line of units out for itself: a few thousand of them at most, a handful per
// thread, which is less than a launch for a plan would take.
template <int ROWS, int STEP, int WAVES>
__device__ __forceinline__ void find_start(const AttnArgs &a, int slots, int slot, int *chunk_s, int *wave_s, int *found_s, Start &st, unsigned &per)
{
    constexpr int kThreads = WAVES * 64;
    const int tid = threadIdx.x, chunk = (a.requests + kThreads - 1) / kThreads;
    const int q0 = min(tid * chunk, a.requests), q1 = min(q0 + chunk, a.requests);
    int tiles = 0, first, n, len, total;
    for (int r = q0; r < q1; ++r) {
        request_of(a, r, first, n, len);
        tiles += tiles_of<ROWS>(a, n);
    }
    const int before = scan<WAVES>(tiles, wave_s, total);
    chunk_s[tid] = before;
    __syncthreads();
    const int share = (total + kThreads - 1) / kThreads, t0 = min(tid * share, total), t1 = min(t0 + share, total);
    // the chunk, then the request, of tile t0
    int r = 0, left = 0;   // left: tiles of r from the current one on
    Unit u{};
    auto locate = [&]() {
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_s[mid] <= t0)
                lo = mid;
            else
                hi = mid;
        }
        r = lo * chunk;
        int t = t0 - chunk_s[lo];
        for (;; ++r) {   // t0 < total: the chunk holds it
            request_of(a, r, u.first, u.n, u.len);
            left = tiles_of<ROWS>(a, u.n);
            if (t < left || r + 1 >= a.requests)
                break;
            t -= left;
        }
        u.tile = t;
        left -= t;
    };
    auto next = [&]() {
        ++u.tile;
        if (--left == 0) {
            while (++r < a.requests) {
                request_of(a, r, u.first, u.n, u.len);
                left = tiles_of<ROWS>(a, u.n);
                if (left)
                    break;
            }
            u.tile = 0;
        }
    };
    int steps = 0;
    if (t0 < t1) {
        locate();
        for (int t = t0; t < t1; ++t) {
            span<ROWS, STEP>(a, u);
            steps += u.steps;
            if (t + 1 < t1)
                next();
        }
    }
    int at = scan<WAVES>(steps, wave_s, st.all);
    // the host has checked that the whole line has less than 2^31 steps
    per = max(((unsigned)st.all * (unsigned)a.kv_heads + (unsigned)slots - 1u) / (unsigned)slots, 1u);
    if (st.all == 0)
        return;
    const int want = (int)((unsigned)slot * per % (unsigned)st.all);
    if (t0 < t1 && at <= want && want < at + steps) {
        locate();
        for (int t = t0; t < t1; ++t) {
            span<ROWS, STEP>(a, u);
            if (want < at + u.steps)
                break;
            at += u.steps;
            next();
        }
        found_s[0] = r;
        found_s[1] = u.tile;
        found_s[2] = want - at;
    }
    __syncthreads();
    st.req = __builtin_amdgcn_readfirstlane(found_s[0]);
    st.tile = __builtin_amdgcn_readfirstlane(found_s[1]);
    st.into = __builtin_amdgcn_readfirstlane(found_s[2]);
}

// ---- a wave's rows ------------------------------------------------------------------
// 32-byte segment c of row r of K or V lies at segment c ^ fold(r) of the row, so that neither the reads of K
// (16 rows of 16 bytes) nor those of V (16 rows of 32 bytes) meet in the same banks.
template <int D>
__device__ __forceinline__ int fold(int row)
{
    return D >= 128 ? row & 7 : (row >> 1) & 3;
}

// 16 keys, one contiguous stretch of a page, to LDS
template <int D>
struct Loader {
    static constexpr int kLoads = D / 32;    // of 1 KB
    static constexpr int kKinds = D >= 256 ? 4 : D >= 128 ? 2 : 1;
    uint32_t off[kKinds];
    __device__ __forceinline__ void init(int lane)
    {
        constexpr int kLanes = D / 8;   // of a row
#pragma unroll
        for (int x = 0; x < kKinds; ++x) {
            const int row = x * (64 / kLanes) + lane / kLanes, c = lane % kLanes;
            off[x] = (uint32_t)(lane / kLanes * D * 2 + (((c >> 1) ^ fold<D>(row)) << 5) + (c & 1) * 16);
        }
    }
    // `from` and `to` are the same in all lanes; lane l's 16 bytes go to to + 16 l. The compiler knows of the load's
    // writes to LDS, but not when they are done: for the builtin it waits for all loads at the next read of
    // any of it by ordinary loads, and never for transposing reads. So this is an asm without outputs, and each
    // read of a buffer stands behind a wait of its own (landed()).
    __device__ __forceinline__ void load(const uint8_t *from, lds_t *to) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                         ::"s"((uint32_t)(uintptr_t)(to + i * 1024)), "v"(off[i % kKinds]), "s"(from + i * 1024)
                         : "memory");   // m0 is the compiler's to set, and it sets it wherever it needs it
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

template <int D, class T, bool EXACT>
struct Rows {
    static constexpr int kQ = D / 32, kO = D / 16, kParts = Split<T, EXACT>::kParts;
    // fp16 weights start at 2^6: small ones keep their bits, and a row whose maximum lags by kLag still fits
    static constexpr float kBias = sizeof(T) && std::is_same<T, F16>::value ? 6.0f : 0.0f, kLag = 8.0f;
    uint4 q[kQ][kParts];
    v4f o[kO];
    float m, base, l, c;  // running maximum of the scores, the same or 0 before there is one, sum of the lane's weights, the scores' factor
    int kmin, kmax;       // keys that the lane's row sees
    uint32_t kread[4], vread[8];

    __device__ __forceinline__ void init_reads(int lane)
    {
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            kread[s] = (uint32_t)(i * D * 2 + ((((2 * s + (g >> 1)) & (D >= 128 ? 7 : 3)) ^ fold<D>(i)) << 5) + (g & 1) * 16);
        const int row = 4 * g + (i >> 2);
#pragma unroll
        for (int d = 0; d < 8; ++d)
            vread[d] = (uint32_t)(row * D * 2 + (((d & (D >= 128 ? 7 : 3)) ^ fold<D>(row)) << 5) + (i & 3) * 8);
    }
    __device__ __forceinline__ uint4 key(const lds_t *buf, int t, int s) const
    {
        constexpr int kPer = D >= 128 ? 4 : 2;   // operands of 256 (or 128) bytes of the row
        return __builtin_bit_cast(uint4, *(const __attribute__((address_space(3))) v4u *)(buf + kread[s % kPer] + s / kPer * 256 + t * 16 * D * 2));
    }
    __device__ __forceinline__ uint4 value(const lds_t *buf, int d) const
    {
        constexpr int kPer = D >= 128 ? 8 : 4;
        uint2 w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            w[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                 (__attribute__((address_space(3))) v4s *)(buf + vread[d % kPer] + d / kPer * 256 + t * 16 * D * 2)));
        return make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    }

    // Row `row` of a unit (rows past the last are that one): its q, and what it sees.
    __device__ __forceinline__ void begin(const AttnArgs &a, const Unit &u, int head, int row, int lane)
    {
        const int r = min(row, u.n * a.group - 1), tok = r / a.group, h = head * a.group + r - tok * a.group, g = lane >> 4;
        const int p = u.len - u.n + tok;
        kmax = max(min(min(u.len, a.width << a.page_shift), p + 1), 0);
        kmin = a.window ? max(p - a.window + 1, 0) : 0;
        const size_t at = (size_t)((long long)(u.first + tok) * a.q_row + (long long)h * a.q_head) + 8 * g;
        c = a.scale;
        if constexpr (!EXACT) {
#pragma unroll
            for (int s = 0; s < kQ; ++s)
                q[s][0] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + at + 32 * s);
        } else {
            Eight<float> e[kQ];
#pragma unroll
            for (int s = 0; s < kQ; ++s)
                e[s].load(static_cast<const float *>(a.q) + at + 32 * s);
            float f = 1.0f;
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
                f = __builtin_ldexpf(1.0f, half);
                const float f2 = __builtin_ldexpf(1.0f, 9 - ex - half);
#pragma unroll
                for (int s = 0; s < kQ; ++s) {
                    e[s].get(v);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        v[x] = v[x] * f * f2;
                    e[s].set(v);
                }
                c = c / f / f2;
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
                        word(q[s][p], x) = w[p];
                }
            }
        }
        // loaded here, or the wait for these loads stands in the loop over the keys, where it would also be one for theirs
#pragma unroll
        for (int s = 0; s < kQ; ++s)
#pragma unroll
            for (int x = 0; x < kParts; ++x)
                asm volatile("" : "+v"(q[s][x].x), "+v"(q[s][x].y), "+v"(q[s][x].z), "+v"(q[s][x].w));
        m = -INFINITY;
        base = 0.0f;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < kO; ++d)
            o[d] = v4f{};
    }

    // Scores of 32 keys from key0 on: s[t][i] is key 16 t + 4 g + i
    __device__ __forceinline__ void scores(const lds_t *kb, v4f (&s)[2]) const
    {
        s[0] = s[1] = v4f{};
        // operands in batches, one on its way while the other is multiplied
        constexpr int kBatch = 4, kBatches = 2 * kQ / kBatch;
        uint4 k[2][kBatch];
        auto read = [&](int b) {
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
                k[b & 1][x] = key(kb, x & 1, (b * kBatch + x) >> 1);
        };
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
                    s[x & 1] = mfma(k[b & 1][x], q[(b * kBatch + x) >> 1][p], s[x & 1], T());
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // `gone`: bit t set where the 16 keys t have no page
    __device__ __forceinline__ bool sees(int key0, int j, int g, uint32_t gone) const
    {
        const int k = key0 + (j >> 2) * 16 + 4 * g + (j & 3);
        return k >= kmin && k < kmax && !(gone >> (j >> 2) & 1);
    }
    __device__ __forceinline__ void hide(int key0, int g, uint32_t gone, v4f (&s)[2]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j >> 2][j & 3] = sees(key0, j, g, gone) ? s[j >> 2][j & 3] : -INFINITY;
    }
    // The weights of 32 keys, and what they do to the maximum and the sum. The maximum follows only when a score
    // exceeds it by kLag: until then weights are larger than one, which costs no bits, and o stays as it is.
    // Scores are subtracted before they are scaled: one fused operation for both would leave the rounding of the
    // maximum's product in the exponent, of any size where scores are large.
    __device__ __forceinline__ void weigh(const v4f (&s)[2], uint4 (&p)[kParts])
    {
        float top = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
        top = fmaxf(top, fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        if (__any((top - m) * c > kLag)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(m, top);
            if (now > m) {
                const float f = __builtin_amdgcn_exp2f((m - now) * c);
                l *= f;
#pragma unroll
                for (int d = 0; d < kO; ++d)
                    o[d] *= f;
                m = base = now;
            }
        }
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j >> 2][j & 3] - base, c, kBias));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            uint32_t parts[kParts];
            Split<T, EXACT>::pair(w[2 * x], w[2 * x + 1], parts);
#pragma unroll
            for (int y = 0; y < kParts; ++y)
                word(p[y], x) = parts[y];
            if constexpr (EXACT)
                l += w[2 * x] + w[2 * x + 1];
            else
                l = dot2(parts[0], ones(T()), l, T());   // the weights as they are used
        }
    }
    __device__ __forceinline__ void add(const lds_t *vb, const uint4 (&p)[kParts])
    {
        constexpr int kBatch = 4, kBatches = kO / kBatch;
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
                    o[b * kBatch + x] = mfma(v[b & 1][x], p[y], o[b * kBatch + x], T());
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The same where some keys are hidden from some rows. A weight of zero does not hide a value that is not
    // finite: keys from `lo` to `hi` are the ones that any row of the unit sees, others are taken for zeros; and
    // if `mixed`, some of these hidden from some rows, keys with such values are added one at a time, to the
    // rows that see them.
    __device__ __forceinline__ void add_some(const lds_t *vb, const uint4 (&p)[kParts], int key0, int g, uint32_t gone, int lo, int hi, bool mixed)
    {
        auto mask_of = [&](uint32_t keys) {   // bit 16 t + k: key k of tile t
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t two = keys >> ((x >> 1) * 16 + 4 * g + (x & 1) * 2);
                w[x] = (two & 1 ? 0xffffu : 0u) | (two & 2 ? 0xffff0000u : 0u);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        auto masked = [&](uint4 v, uint4 k) { return make_uint4(v.x & k.x, v.y & k.y, v.z & k.z, v.w & k.w); };
        // keys lo .. hi - 1 as bits
        auto low_bits = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
        uint32_t keep = low_bits(hi - key0) & ~low_bits(lo - key0);
        keep &= ~((gone & 1 ? 0xffffu : 0u) | (gone & 2 ? 0xffff0000u : 0u));
        uint32_t strange = 0;   // bit j: the lane's key j has a value that is not finite
        if (mixed) {
            const uint4 k = mask_of(keep);
#pragma unroll 2
            for (int d = 0; d < kO; ++d) {
                const uint4 v = masked(value_at(vb, d), k);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    constexpr uint32_t e = exponents(T());
                    strange |= ((w[x] & e & 0xffffu) == (e & 0xffffu) ? 1u << (2 * x) : 0u) |
                               ((w[x] & e & 0xffff0000u) == (e & 0xffff0000u) ? 2u << (2 * x) : 0u);
                }
            }
        }
        uint32_t apart = 0;
        if (__any(strange)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const unsigned long long set = __ballot(strange >> j & 1);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    apart |= (set >> (16 * x) & 0xffffu) ? 1u << ((j >> 2) * 16 + 4 * x + (j & 3)) : 0u;
            }
        }
        const uint4 k = mask_of(keep & ~apart);
#pragma unroll
        for (int d = 0; d < kO; ++d) {
            const uint4 v = masked(value(vb, d), k);
#pragma unroll
            for (int y = kParts; y-- > 0;)
                o[d] = mfma(v, p[y], o[d], T());
        }
        while (apart) {
            const int one = __builtin_ctz(apart);
            apart &= apart - 1;
            const uint4 ko = mask_of(1u << one);
            const int kk = key0 + one;
            const bool seen = kk >= kmin && kk < kmax;
#pragma unroll
            for (int d = 0; d < kO; ++d) {
                const uint4 v = masked(value(vb, d), ko);
                v4f x = o[d];
#pragma unroll
                for (int y = kParts; y-- > 0;)
                    x = mfma(v, p[y], x, T());
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[d][i] = seen ? x[i] : o[d][i];
            }
        }
    }
    // value() of a d that is not known at compile time
    __device__ __forceinline__ uint4 value_at(const lds_t *buf, int d) const
    {
        constexpr int kPer = D >= 128 ? 8 : 4;
        const uint32_t at = (vread[0] ^ ((uint32_t)(d % kPer) << 5)) + d / kPer * 256;
        uint2 w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            w[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)(buf + at + t * 16 * D * 2)));
        return make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    }
    // the row's sum, in all four lanes that share it
    __device__ __forceinline__ void end()
    {
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
    }
};

// ---- results ------------------------------------------------------------------------
// o[0..3] / l, gated, as elements d .. d + 3 of the unit's row `row`
template <class Q, int D>
__device__ __forceinline__ void put_out(const AttnArgs &a, int first, int group_row, int head, int d, v4f o, float l)
{
    const int tok = group_row / a.group, h = head * a.group + group_row - tok * a.group;
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
constexpr int kNarrowWaves = 4, kNarrowRows = 16, kNarrowStep = kNarrowWaves * kBlk;

// workgroups of a CU: what LDS holds (128, 64 or 32 KB each), and registers
constexpr int narrow_per_cu(int dim) { return dim == 256 ? 1 : dim == 128 ? 2 : 3; }

template <int D, class T, class Q>
__global__ __launch_bounds__(kNarrowWaves * 64, narrow_per_cu(D)) void attn_narrow_kernel(AttnArgs a)
{
    constexpr bool kExact = std::is_same<Q, float>::value;
    using R = Rows<D, T, kExact>;
    constexpr int kBuf = kBlk * D * 2;
    // arrays of their own: a read of one then waits for no load of the other
    __shared__ __align__(128) uint8_t kbuf[kNarrowWaves * kBuf];
    __shared__ __align__(128) uint8_t vbuf[kNarrowWaves * kBuf];
    __shared__ int chunk_s[kNarrowWaves * 64];
    __shared__ int wave_s[kNarrowWaves], found_s[3];
    __shared__ float m_s[kNarrowWaves][kNarrowRows], l_s[kNarrowWaves][kNarrowRows], c_s[kNarrowRows];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
    // neighbours on the line of units share keys: they go to the same XCD (workgroup b runs on XCD b % 8)
    const int slots = gridDim.x, slot = (int)(blockIdx.x & 7) * (slots >> 3) + (int)(blockIdx.x >> 3);
    Start st;
    unsigned per;
    find_start<kNarrowRows, kNarrowStep, kNarrowWaves>(a, slots, slot, chunk_s, wave_s, found_s, st, per);
    unsigned line = (unsigned)slot * per;
    const unsigned end = min(line + per, (unsigned)st.all * (unsigned)a.kv_heads);
    Meta *meta = reinterpret_cast<Meta *>(a.meta) + slot;
    int parts = 0;
    if (line < end) {
        lds_t *kb = (lds_t *)kbuf + wave * kBuf, *vb = (lds_t *)vbuf + wave * kBuf;
        const const_ints table = (const_ints)a.table;
        int head = (int)(line / (unsigned)st.all), req = st.req, into = st.into;
        Unit u;
        u.tile = st.tile;
        Loader<D> loader;
        loader.init(lane);
        R rows;
        rows.init_reads(lane);
        for (;;) {
            request_of(a, req, u.first, u.n, u.len);
            u.first = __builtin_amdgcn_readfirstlane(u.first);
            u.n = __builtin_amdgcn_readfirstlane(u.n);
            u.len = __builtin_amdgcn_readfirstlane(u.len);
            span<kNarrowRows, kNarrowStep>(a, u);
            const int take = (int)min((unsigned)(u.steps - into), end - line);
            const int row0 = u.tile * kNarrowRows, nrows = min(u.n * a.group - row0, kNarrowRows);

            // all rows see keys from some_lo on up to some_hi; any row, those from kbeg on up to kend
            int some_lo = 0, some_hi;
            {
                const int p0 = u.len - u.n + row0 / a.group, p1 = u.len - u.n + (row0 + nrows - 1) / a.group;
                some_hi = max(min(u.kend, p0 + 1), 0);
                if (a.window)
                    some_lo = max(p1 - a.window + 1, 0);
            }
            const int hi = min((u.s0 + into + take) * kNarrowStep, u.kend);
            int blk = (u.s0 + into) * kNarrowWaves + wave;
            while ((blk + 1) * kBlk <= u.kbeg)
                blk += kNarrowWaves;
            // the 16 keys from `key` on: their page's address, or 0 and a set bit in `gone`
            auto place = [&](int key, int t, uint32_t &gone) {
                int id = -1;
                if (key < u.kend)
                    id = table[(size_t)req * a.width + (key >> a.page_shift)];
                if ((unsigned)id >= (unsigned)a.pages) {
                    gone |= 1u << t;
                    id = 0;
                }
                return ((((size_t)id * a.kv_heads + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * (D * 2);
            };
            size_t at[2];
            uint32_t gone = 0;
            if (blk * kBlk < hi) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    at[t] = place(blk * kBlk + 16 * t, t, gone);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    loader.load(a.k + at[t], kb + t * 16 * D * 2);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    loader.load(a.v + at[t], vb + t * 16 * D * 2);
            }
            rows.begin(a, u, head, row0 + i, lane);   // behind the loads of keys and values: waited for once, with them
            while (blk * kBlk < hi) {
                const int key0 = blk * kBlk, next = blk + kNarrowWaves;
                const bool more = next * kBlk < hi;
                size_t nat[2] = {0, 0};
                uint32_t ngone = 0;
                if (more) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        nat[t] = place(next * kBlk + 16 * t, t, ngone);
                }
                v4f s[2];
                landed<2 * Loader<D>::kLoads>();   // all but the values, which were asked for last
                rows.scores(kb, s);
                lds_read();
                if (more) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        loader.load(a.k + nat[t], kb + t * 16 * D * 2);
                }
                if (more)   // the next keys may be on their way
                    landed<2 * Loader<D>::kLoads>();
                else
                    landed<0>();
                const bool whole = key0 >= some_lo && key0 + kBlk <= some_hi && !gone;
                if (!whole)
                    rows.hide(key0, g, gone, s);
                uint4 p[R::kParts];
                rows.weigh(s, p);
                if (whole)
                    rows.add(vb, p);
                else
                    rows.add_some(vb, p, key0, g, gone, u.kbeg, u.kend,
                                  min(key0 + kBlk, u.kend) > some_hi || max(key0, u.kbeg) < some_lo);
                lds_read();
                if (more) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        loader.load(a.v + nat[t], vb + t * 16 * D * 2);
                }
                gone = ngone;
                blk = next;
            }
            rows.end();

            // the waves' sums become one, in the order of the waves
            if (g == 0) {
                m_s[wave][i] = rows.m;
                l_s[wave][i] = rows.l;
                c_s[i] = rows.c;   // the same in all waves
            }
            __syncthreads();
            float top = m_s[0][i];
#pragma unroll
            for (int w = 1; w < kNarrowWaves; ++w)
                top = fmaxf(top, m_s[w][i]);
            const float f = rows.m == top ? 1.0f : __builtin_amdgcn_exp2f((rows.m - top) * rows.c);
            float *mine = reinterpret_cast<float *>(kbuf) + wave * kNarrowRows * D;
#pragma unroll
            for (int d = 0; d < R::kO; ++d)
                *reinterpret_cast<v4f *>(mine + i * D + ((4 * d + g) ^ i) * 4) = rows.o[d] * f;
            __syncthreads();
            const bool begins = into == 0, ends = into + take == u.steps;
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
                    o += *reinterpret_cast<const v4f *>(reinterpret_cast<const float *>(kbuf) + (w * kNarrowRows + r) * D + (ch ^ r) * 4);
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
                // its last step is step line + steps - 1 of the line
                parts = (int)((line + (unsigned)u.steps - 1u) / per) - slot + 1;
                if (tid == 0)
                    *meta = Meta{parts, head, u.first, u.n * a.group, row0, {}};
            }
            line += take;
            if (line >= end)
                break;
            // the next unit
            into = 0;
            ++u.tile;
            if (u.tile * kNarrowRows >= u.n * a.group) {
                u.tile = 0;
                int first, n, len;
                do {
                    if (++req == a.requests) {
                        req = 0;
                        ++head;
                    }
                    request_of(a, req, first, n, len);
                } while (__builtin_amdgcn_readfirstlane(n) == 0);   // line < end: there is one
            }
            __syncthreads();
        }
    }
    if (parts == 0 && tid == 0)
        meta->parts = 0;
}

// ---- units that a border cut ---------------------------------------------------------
// Workgroup (slot, y) joins 1024 / D rows of the unit that begins in the slot, if it ends in another:
// o = sum_j 2^(c (m_j - m)) o_j and l likewise, over the parts in order.
template <int ROWS, int D, class Q>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a)
{
    constexpr int kRows = 1024 / D, kLanes = D / 4;   // rows of a workgroup, threads of a row
    const int slot = blockIdx.x, r = blockIdx.y * kRows + threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
    const Meta meta = reinterpret_cast<const Meta *>(a.meta)[slot];
    if (meta.parts == 0 || meta.row0 + r >= meta.rows)
        return;
    const float *first = part_of<ROWS, D>(a, slot, true);
    const float *others = part_of<ROWS, D>(a, slot + 1, false);
    constexpr size_t kNext = 2 * ROWS * (D + 3);
    const float c = first[ROWS * D + 2 * ROWS + r];
    float best = first[ROWS * D + r];
    for (int j = 1; j < meta.parts; ++j)
        best = fmaxf(best, others[(j - 1) * kNext + ROWS * D + r]);
    v4f o = {};
    float l = 0.0f;
    for (int j = 0; j < meta.parts; ++j) {
        const float *p = j ? others + (j - 1) * kNext : first;
        const float m = p[ROWS * D + r], f = m == best ? 1.0f : __builtin_amdgcn_exp2f((m - best) * c);
        o += *reinterpret_cast<const v4f *>(p + r * D + d) * f;
        l += p[ROWS * D + ROWS + r] * f;
    }
    put_out<Q, D>(a, meta.first, meta.row0 + r, meta.head, d, o, l);
}

// ---- host ---------------------------------------------------------------------------
// As many workgroups as the chip's 256 CUs hold at a time: a constant, as the order of the sums must not depend
// on a partition's size.
int slots_of(int dim) { return 256 * narrow_per_cu(dim); }
constexpr size_t kMetaBytes = 768 * sizeof(Meta);

size_t workspace(int dim) { return kMetaBytes + (size_t)slots_of(dim) * 2 * kNarrowRows * (dim + 3) * 4; }

template <int D, class T, class Q>
int launch(const AttnArgs &a, hipStream_t st)
{
    const int slots = slots_of(D);
    hipLaunchKernelGGL((attn_narrow_kernel<D, T, Q>), dim3(slots), dim3(kNarrowWaves * 64), 0, st, a);
    if (hipGetLastError() != hipSuccess)
        return TB_EHIP;
    hipLaunchKernelGGL((attn_join_kernel<kNarrowRows, D, Q>), dim3(slots, kNarrowRows * D / 1024), dim3(256), 0, st, a);
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

extern "C" size_t tb_attn_paged_workspace_bytes(const tb_kv_cache *cache, int heads, int dtype, int requests, int tokens)
{
    if (!cache || !shapes_ok(*cache, heads, dtype, requests, tokens) || !runs(*cache, heads, requests, tokens))
        return 0;
    return workspace(cache->dim);
}

extern "C" int tb_attn_paged(const tb_heads *q, const tb_heads *gate, const tb_kv_cache *cache, const int32_t *table, int width,
                             const int32_t *offsets, const int32_t *lengths, int requests, int tokens, float scale, int window,
                             void *out, void *ws, size_t ws_bytes, void *stream)
{
    if (!q || !cache || !shapes_ok(*cache, q->heads, q->dtype, requests, tokens) || width < 1 || window < 0 || !(scale > 0.0f) || scale > 3.0e38f)
        return TB_EINVAL;
    const int dim = cache->dim;
    if (gate && gate->heads != q->heads)
        return TB_EINVAL;
    const size_t qb = tbh::heads_bytes(*q, tokens, dim), gb = gate ? tbh::heads_bytes(*gate, tokens, dim) : 0;
    if (!qb || (gate && !gb))
        return TB_EINVAL;
    const bool can = runs(*cache, q->heads, requests, tokens);
    const size_t need = can ? workspace(dim) : 0;
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
    // steps of all units are counted in 31 bits
    if (!can || limit > (1 << 30) ||
        ((long long)tokens * q->heads / 16 + (long long)requests * cache->kv_heads) * (limit / 64 + 2) >= (1ll << 31))
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
    r.group = q->heads / cache->kv_heads, r.requests = requests, r.tokens = tokens;
    r.window = std::min(window, 1 << 30), r.scale = scale * kLog2e, r.out = out;
    r.meta = static_cast<int32_t *>(ws), r.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kMetaBytes);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (cache->dtype == TB_BF16)
        return q->dtype == TB_F32 ? launch_dim<Bf16, float>(dim, r, st) : launch_dim<Bf16, Bf16>(dim, r, st);
    return q->dtype == TB_F32 ? launch_dim<F16, float>(dim, r, st) : launch_dim<F16, F16>(dim, r, st);
}
