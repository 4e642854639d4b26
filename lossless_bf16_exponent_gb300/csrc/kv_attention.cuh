// kv_attention.cuh -- what the attention and mass kernels share: parameters,
// the split of the cache's tiles over the grid, masks, and the warp-level
// matrix products on 16-bit and E5M2 rows in shared memory.
//
// Rows. The group's query heads of all new tokens of one (sequence, KV head)
// are rows of one product: row r is token r / group, head r % group, so a
// cached row is read once for all of them.
//
// E5M2 rows stay bytes in shared memory. E5M2 is the upper byte of FP16, so a
// byte permute widens two of them to a pair that the FP16 product takes.
#pragma once

#include <type_traits>

#include "kv_index.cuh"
#include "kv_internal.cuh"

namespace uzkv {

constexpr uint32_t kMaxAttGrid = 160;   // bounds the workspace; one CTA an SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttParams {
    Rows q, out;
    float* lse;
    const int64_t* mask;
    int64_t mask_b;
    uint32_t mask_words;
    const int32_t* counts;
    const float* weights;
    Cache cache;
    float scale;
    uint32_t tokens, q_heads, group;
    uint32_t rows;     // tokens * group
    uint32_t mtiles;   // row tiles of a (sequence, KV head)
    uint32_t m;        // rows of a tile
    uint32_t dp;       // floats a row of a partial result takes
    uint32_t grid;     // CTAs the tiles are split over
    uint32_t shift;    // log2 of the cached tokens of a tile
    uint32_t unit_cost;  // tiles that a unit weighs beyond its own
    float* partial;    // [grid][2] results: m rows of dp floats, then m (reference, sum) pairs
    const float* mass_in;
    float* mass_out;
    float decay;
    int64_t mass_b, mass_h;
    uint32_t slots;
};

__device__ __forceinline__ uint64_t partial_floats(const AttParams& p) { return (uint64_t)p.m * (p.dp + 2); }

// ------------------------------------------------------------------- split
//
// The tiles of all (sequence, KV head, row tile) units in this order, cut into
// equal runs, one a CTA: sequences of any lengths load all SMs alike. Each unit
// has `unit_cost` positions before its tiles, which stand for the time of its
// queries' load and its output, so that many short units weigh as much as they
// take. A unit that several CTAs share leaves partial results: a CTA's first
// unit in its slot 0 where the unit began before it, its last unit in slot 1
// where the unit goes on after it.

struct Unit {
    uint32_t b, h, mt, tile, tiles;
    Span span;
    uint64_t pos;  // position of the tile
};

__device__ __forceinline__ uint32_t tiles_of(const AttParams& p, const Span& s) {
    return s.fresh ? (s.old + s.fresh + (1u << p.shift) - 1) >> p.shift : 0;
}

__device__ __forceinline__ uint32_t tiles_of(const AttParams& p, uint32_t b) {
    return b < p.cache.sequences ? tiles_of(p, span_of(p.cache, p.counts, p.tokens, b)) : 0;
}

// Positions that a unit of so many tiles takes.
__device__ __forceinline__ uint32_t width_of(const AttParams& p, uint32_t tiles) { return tiles ? tiles + p.unit_cost : 0; }

// What a warp knows of the split: the positions of all sequences (one head and row tile each), and of sequence `lane`.
struct Split {
    uint64_t all;
    uint32_t mine;
};

// All lanes of a warp.
__device__ __forceinline__ Split split_of(const AttParams& p) {
    const uint32_t lane = threadIdx.x % 32;
    Split s;
    s.mine = width_of(p, tiles_of(p, lane));
    s.all = s.mine;
    for (uint32_t b = lane + 32; b < p.cache.sequences; b += 32) s.all += width_of(p, tiles_of(p, b));
    for (int o = 16; o; o >>= 1) s.all += __shfl_xor_sync(0xFFFFFFFFu, s.all, o);
    return s;
}

// All lanes of a warp: the first unit and tile at or after position `at` of the order, at < all * kv_heads * mtiles.
__device__ __forceinline__ Unit unit_at(const AttParams& p, const Split& s, uint64_t at, uint32_t mtiles) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t per = (uint64_t)p.cache.kv_heads * mtiles;
    uint64_t before = 0;
    Unit u{};
    for (uint32_t b0 = 0; b0 < p.cache.sequences; b0 += 32) {
        const uint64_t mine = b0 ? width_of(p, tiles_of(p, b0 + lane)) : s.mine;
        uint64_t upto = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= (uint32_t)o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, (before + upto) * per > at);
        if (past) {
            const int l = __ffs(past) - 1;
            const uint64_t start = __shfl_sync(0xFFFFFFFFu, before + upto - mine, l) * per;
            const uint32_t width = (uint32_t)__shfl_sync(0xFFFFFFFFu, mine, l);
            u.b = b0 + l;
            u.tiles = width - p.unit_cost;
            const uint64_t in = at - start;  // within one sequence
            const uint32_t unit = (uint32_t)divide(in, width), off = (uint32_t)(in - (uint64_t)unit * width);
            u.tile = off > p.unit_cost ? off - p.unit_cost : 0;
            u.pos = at + (off < p.unit_cost ? p.unit_cost - off : 0);
            u.h = unit / mtiles;
            u.mt = unit - u.h * mtiles;
            u.span = span_of(p.cache, p.counts, p.tokens, u.b);
            return u;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    u.pos = ~0ull;
    return u;
}

// On to the next tile.
__device__ __forceinline__ void advance(const AttParams& p, Unit& u, uint32_t mtiles) {
    u.pos++;
    if (++u.tile < u.tiles) return;
    u.tile = 0;
    u.pos += p.unit_cost;
    if (++u.mt < mtiles) return;
    u.mt = 0;
    if (++u.h < p.cache.kv_heads) return;
    u.h = 0;
    do {
        if (++u.b >= p.cache.sequences) {
            u.pos = ~0ull;
            return;
        }
        u.span = span_of(p.cache, p.counts, p.tokens, u.b);
        u.tiles = tiles_of(p, u.span);
    } while (!u.tiles);
}

// A CTA's run of positions.
struct Run {
    uint64_t begin, end;
};
__device__ __forceinline__ Run run_of(const AttParams& p, const Split& s, uint32_t mtiles) {
    const uint64_t total = s.all * p.cache.kv_heads * mtiles, shares = min(total, (uint64_t)p.grid);  // no share is empty
    if (blockIdx.x >= shares) return Run{0, 0};
    if (total * shares >> 32 == 0) {  // the common case, without 64-bit division
        const uint32_t t = (uint32_t)total, n = (uint32_t)shares;
        return Run{t * blockIdx.x / n, t * (blockIdx.x + 1) / n};
    }
    return Run{total * blockIdx.x / shares, total * (blockIdx.x + 1) / shares};
}

// ------------------------------------------------------------------- masks

// Which of the slots j0 .. j0 + 63 row r sees, as bits.
__device__ __forceinline__ uint64_t seen_bits(const AttParams& p, uint32_t b, const Span& s, uint32_t row, uint32_t j0) {
    const uint32_t t = row / p.group;
    if (row >= p.rows || t >= s.fresh) return 0;
    const int64_t u0 = (int64_t)j0 - s.old;
    if (u0 <= -64) return ~0ull;
    const int64_t* w = p.mask ? p.mask + b * p.mask_b + (uint64_t)t * p.mask_words : nullptr;
    auto word = [&](uint32_t i) -> uint64_t {
        if (w) return i < p.mask_words ? (uint64_t)w[i] : 0;
        const int32_t n = (int32_t)t + 1 - (int32_t)(64 * i);  // a chain: bits 0 .. t
        return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
    };
    uint64_t bits;
    if (u0 < 0) {
        bits = ((1ull << -u0) - 1) | word(0) << -u0;
    } else {
        const uint32_t i = (uint32_t)u0 / 64, o = (uint32_t)u0 % 64;
        bits = word(i) >> o;
        if (o) bits |= word(i + 1) << (64 - o);
    }
    const int64_t live = (int64_t)s.fresh - u0;  // slots from j0 on that are in use
    return live >= 64 ? bits : live <= 0 ? 0 : bits & ((1ull << live) - 1);
}

// --------------------------------------------------------------- PTX pieces

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory; zeros where !valid.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// An 8 x 8 matrix of 16-bit elements across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

// 2^x with a relative error up to 2^-22; results below 2^-126 are zero. Both are far below a weight's 16 bits, and the
// largest weight of a row is at least 1 here.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Whether the phase of the given parity has ended.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done;
}
// Waits for the phase of the given parity to end. Bounded: false after about a second, which only a fault in the
// kernel's own counting could bring about; the caller then leaves its loop.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < (1u << 20); i++) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}
// The same for a whole warp, which stays together whatever the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity)); }

// One arrival once this thread's copies so far have landed; counted among the barrier's own.
__device__ __forceinline__ void bar_arrive_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Eight E5M2 bytes to FP16.
__device__ __forceinline__ uint4 widen(uint32_t a, uint32_t b) {
    return make_uint4(uzip::prmt(a, 0, 0x1404), uzip::prmt(a, 0, 0x3424), uzip::prmt(b, 0, 0x1404), uzip::prmt(b, 0, 0x3424));
}

// NaN and infinities of a pair of values (FP16 or BF16 patterns) become zero; whether there were any.
template <typename T>
__device__ __forceinline__ uint32_t clean2(uint32_t& v) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    uint32_t bad = 0;
    if ((v & kExp) == kExp) bad |= 0xFFFFu;
    if ((v >> 16 & kExp) == kExp) bad |= 0xFFFF0000u;
    v &= ~bad;
    return bad;
}

// Byte offset of 16-byte chunk c of row r in a shared-memory tile of `rows` rows of RB bytes: blocks of 128 bytes a
// row one after the other (or the 64 that a row has), chunks XORed with the row so that the eight rows of a matrix
// load lie in eight bank groups. This is the accelerator's own 128-byte (64-byte) swizzle, and the tensor core's.
template <int RB>
__device__ __forceinline__ uint32_t row_chunk(uint32_t rows, uint32_t r, uint32_t c) {
    static_assert(RB == 64 || RB == 128 || RB == 256 || RB == 512, "row bytes");
    return RB == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Weights go to the 16-bit product as exp2(x - reference), and the reference may trail the running maximum by
// kSlack before a row is rescaled, so that most steps need neither the maximum over the warp nor the rescaling.
// FP16, whose largest number is below 2^16 and whose smallest normal one is 2^-14, has the reference 2^6 below the
// maximum it was taken from: weights up to 2^14. BF16 has the range of FP32.
constexpr float kSlack = 8.0f;
template <typename T>
constexpr float kLift = 0.0f;
template <>
constexpr float kLift<__half> = 6.0f;

// BF16 queries of an FP16 product (an E5M2 cache): a power of two is taken out of each row and put back on its scores.
// It brings the row's largest element `top` to [1, 2), to [2, 4) from 2^127 on, and below 1 where top is subnormal: both
// powers are normal numbers, and neither end of BF16's range passes FP16's. BF16's eight bits fit FP16's eleven down to
// 2^-14; smaller elements are rounded to multiples of 2^-24, so a score is off by at most 2^-24 top * sum |k|, about
// what the product's 32-bit sums round away beside a term of the largest element.
struct RowScale {
    float down, up;
    __device__ __forceinline__ explicit RowScale(float top) {
        const uint32_t ex = top == 0.0f ? 127u : min(max(__float_as_uint(top) >> 23, 1u), 253u);  // 127: nothing to scale
        down = __uint_as_float((254 - ex) << 23);
        up = __uint_as_float(ex << 23);
    }
};

// Queries of rows row0 .. row0 + rows - 1 to shared memory as T (columns past head_dim and rows past p.rows
// zero), by THREADS threads numbered tid; at(row, c) is where 16-byte chunk c of a row goes. factor[r] is what a
// score of row r is to be multiplied by to have it in units of log2: |scale| * log2(e), and for BF16 queries that
// go to an FP16 product the power of two that was taken out of the row.
// The sign of scale goes to the queries.
template <typename QT, typename T, int DP, int THREADS, typename At>
__device__ __forceinline__ void load_queries(const AttParams& p, uint32_t tid, uint32_t b, uint32_t h, uint32_t row0,
                                             uint32_t rows, At at, float* factor) {
    constexpr bool kCast = !std::is_same<QT, T>::value;
    constexpr uint32_t kChunks = DP / 8;  // a power of two, at most 32
    const uint32_t c = tid % kChunks, live = p.cache.head_dim / 8;
    constexpr int kBatch = 8;  // rows on their way at once
    constexpr uint32_t kStep = THREADS / kChunks;
    for (uint32_t i0 = tid / kChunks; i0 < rows; i0 += kStep * kBatch) {
        uint4 in[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const uint32_t row = row0 + i0 + k * kStep;
            in[k] = make_uint4(0, 0, 0, 0);
            if (i0 + k * kStep < rows && row < p.rows && c < live) {
                const uint32_t t = row / p.group, g = row - t * p.group;
                in[k] = *reinterpret_cast<const uint4*>(p.q.p + b * p.q.b + t * p.q.t + (uint64_t)(h * p.group + g) * p.q.h + c * 16);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
            const uint32_t i = i0 + k * kStep;
            if (i >= rows) break;  // rows is a multiple of 16 and so of what a pass takes: all lanes of a warp alike
            uint4 x = in[k];
            float f = fabsf(p.scale) * kLog2e;
            if (kCast) {
                const QT* e = reinterpret_cast<const QT*>(&x);
                float v[8], top = 0.0f;
#pragma unroll
                for (int y = 0; y < 8; y++) {
                    v[y] = to_f32(e[y]);
                    top = fmaxf(top, fabsf(v[y]));
                }
                for (uint32_t o = kChunks / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const RowScale row(top);
                f *= row.up;
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                for (int y = 0; y < 4; y++) w[y] = pack2<__half>(v[2 * y] * row.down, v[2 * y + 1] * row.down);
            }
            if (p.scale < 0.0f) {
                x.x ^= 0x80008000u;
                x.y ^= 0x80008000u;
                x.z ^= 0x80008000u;
                x.w ^= 0x80008000u;
            }
            *at(i, c) = x;
            if (c == 0) factor[i] = f;
        }
    }
}

// Attention kernels by types, one translation unit each; they set p.m, p.mtiles, p.dp and p.grid.
int attend_bf16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_bf16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_fp16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_fp16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_many_bf16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);  // more rows, heads up to 128
int attend_many_bf16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_many_fp16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int attend_many_fp16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int mass_bf16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int mass_bf16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int mass_fp16(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);
int mass_fp16_e5m2(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s);

}  // namespace uzkv
