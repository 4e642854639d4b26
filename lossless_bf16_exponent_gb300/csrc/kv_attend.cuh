// kv_attend.cuh -- attention over a paged cache by warp-level matrix products,
// for few rows (or heads above 128): one pass over keys and values with the running
// reference and sum of a softmax.
//
// Bound: HBM, as long as the products of a tile take less time than its bytes
// (4 D flop a row and token against 2 D elements' bytes: up to about 32 rows at
// the warp-level product's rate). So the kernel is built to keep
// copies in flight: one CTA an SM, four warps that only copy, 16 bytes a thread
// and instruction (bulk tensor copies measured no better here: 241 / 242 us at
// pages of 64 tokens, 159 / 120 us for E5M2 heads of 64), eight that only compute,
// and a ring of stages between them. The copies' pages are looked up one tile
// ahead, and the ring runs on across unit boundaries.
//
// The products have the cached tokens along M: S^T = K Q^T and O^T = V^T P^T,
// 16 tokens (or 16 columns of V) by 8 rows. Eight rows of a decoding step waste
// nothing, keys and values are the operand that one matrix load brings whole,
// queries stay in registers, and a score tile becomes the second product's
// operand by one 8 x 8 transpose. A warp takes 8 RN rows; WM warps share the
// rows of a tile and 8 / WM its tokens, which are merged once a unit through
// shared memory.
//
// Measured: 8 rows of 128 over 40 sequences of up to 16,384 tokens (1.6 GB), pages of 16: 240 us, 6.68 TB/s, 98 % of
// the measured copy rate; heads of 64 134 us (88 %); E5M2 of 128 159 us, of 64 118 us, where widening and the
// products' instructions take longer than the bytes; 32 rows of 128 323 us (82 %).
//
// E5M2: a matrix load of 16-bit units gives a thread four consecutive bytes of
// a key row, where the product's layout wants two pairs eight apart. The sum
// over the head dimension may run in any order, so the queries are read in the
// same permuted one. For the values, a transposed load gives the bytes of two
// neighbouring columns; the even ones become rows 0-7 of the product, the odd
// ones rows 8-15.
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_attention.cuh"

namespace uzkv {

template <typename QT, bool FP8, int DP, int RN, int WM>
struct AttCfg {
    using T = typename std::conditional<FP8, __half, QT>::type;  // type of the products
    static constexpr int kRB = DP * (FP8 ? 1 : 2);               // bytes of a cached row in shared memory
    static constexpr int kM = 8 * RN * WM;                       // rows of a unit
    static constexpr int kWN = 8 / WM;
    static constexpr int kTile = kRB == 512 ? 64 : 128;          // cached tokens of a stage
    static constexpr int kKeys = kTile / kWN;                    // of them, a warp's
    static constexpr int kSub = kKeys < 32 ? kKeys : 32;         // taken at once
    static constexpr int kStage = 2 * kTile * kRB;
    static constexpr int kBoxRow = DP + 4;                       // floats; 4 more keep the merge's stores off each other's banks
    static constexpr int kBox = 8 * 8 * kBoxRow * 4;             // eight rows of each computing warp
    static constexpr int kOther = kBox + 8 * 8 * 8 + 256;        // (reference, sum) pairs, barriers
    static constexpr int kFit = (227 * 1024 - kOther) / kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kSmem = kStages * kStage + kOther;
    static_assert(kStages >= 2, "a tile in use and one on its way");
    static_assert(kKeys >= 16, "a product's tokens");
};

constexpr int kAttThreads = 12 * 32;  // 8 warps that compute, 4 that copy

// The launch's 384 x 168 registers, shared out anew: 4 warps x 32 x 72 + 8 x 32 x 216 are as many.
template <bool COMPUTES>
__device__ __forceinline__ void registers() {
    if (COMPUTES) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
}

template <typename QT, bool FP8, int DP, int RN, int WM>
__global__ void __launch_bounds__(kAttThreads, 1) attend_kernel(const __grid_constant__ AttParams p) {
    using C = AttCfg<QT, FP8, DP, RN, WM>;
    using T = typename C::T;
    extern __shared__ __align__(1024) char smem[];
    float* const box = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
    float2* const stat = reinterpret_cast<float2*>(box + 8 * 8 * C::kBoxRow);  // [8 warps][8 rows]
    const uint32_t full = smem_u32(stat + 64), freed = full + 8 * 8, merge = full + 16 * 8;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, l = lane % 4;
    const uint32_t D = p.cache.head_dim;

    uzip::pdl_launch_dependents();
    if (tid == 0) {
        for (int s = 0; s < C::kStages; s++) {
            bar_init(full + 8 * s, 128);  // every copying thread
            bar_init(freed + 8 * s, 8);   // every computing warp
        }
        bar_init(merge, 8);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (D < DP)  // columns past the head dimension stay zero: no copy writes them
        for (uint32_t i = tid; i < C::kStages * C::kStage / 16; i += kAttThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    const Split split = split_of(p);
    const Run run = run_of(p, split, p.mtiles);
    Unit cur{};
    cur.pos = ~0ull;
    if (run.begin != run.end) cur = unit_at(p, split, run.begin, p.mtiles);
    __syncthreads();
    bool ok = true;

    if (warp >= 8) {
        registers<false>();
        // ---- copies: a warp takes a quarter of a tile's tokens
        constexpr uint32_t kMine = C::kTile / 4, kLanes = C::kRB / 16;
        const uint32_t w = warp - 8, c = lane % kLanes, live = D * (FP8 ? 1 : 2) / 16;
        Place at{0, 0};
        bool used = false;  // whether there is such a token
        auto find = [&]() {  // this lane's token of the tile under `cur`
            Place pl{0, 0};
            const uint32_t j = cur.tile * C::kTile + w * kMine + lane;
            used = cur.pos < run.end && lane < kMine && j < cur.span.old + cur.span.fresh;
            if (used) pl = look_up(p.cache, cur.b, j);
            return pl;
        };
        at = find();
        for (uint32_t i = 0; cur.pos < run.end && ok; i++) {
            const Place now = used ? checked(p.cache, at) : Place{-1, 0};
            const char* krow = now.page >= 0 ? k_row(p.cache, now, cur.h) : nullptr;
            const char* vrow = now.page >= 0 ? v_row(p.cache, now, cur.h) : nullptr;
            advance(p, cur, p.mtiles);
            at = find();
            const uint32_t s = i % C::kStages;
            if (i >= C::kStages) ok = warp_wait(freed + 8 * s, (i / C::kStages - 1) & 1);
            if (!ok) break;
            const uint32_t ks = smem_u32(smem + s * C::kStage);
#pragma unroll 8
            for (uint32_t x = 0; x < kMine * kLanes / 32; x++) {
                const uint32_t r = x * (32 / kLanes) + lane / kLanes;
                const char* ka = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(krow), r));
                const char* va = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(vrow), r));
                const uint32_t dst = ks + row_chunk<C::kRB>(C::kTile, w * kMine + r, c);
                if (c < live) {
                    copy16(dst, ka ? ka + c * 16 : p.cache.k, ka != nullptr);
                    copy16(dst + C::kTile * C::kRB, va ? va + c * 16 : p.cache.v, va != nullptr);
                }
            }
            bar_arrive_copies(full + 8 * s);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ---- products
        registers<true>();
        const uint32_t wm = warp % WM, wn = warp / WM, mykey = wn * C::kKeys;
        uint32_t q[RN][DP / 16][2];
        float o[DP / 16][RN][4], f[RN][2], ref[RN][2], sum[RN][2];  // rows 2 l and 2 l + 1 of each tile of eight
        uint32_t merges = 0, first = 0;  // first: the tile with which this CTA began the unit
        bool begun = false;
        // Column of o[x][.][y]: x * 16 + g + 8 (y / 2), or with the even and odd columns apart.
        // The address 32 bytes of a row further on, `i` times: blocks of 128 bytes lie a tile's rows apart.
        auto step_of = [](uint32_t base, uint32_t i) { return (base + (i >> 2) * C::kTile * 128) ^ ((i & 3) << 5); };
        auto column = [&](int x, int y) { return x * 16 + (FP8 ? 2 * g + y / 2 : g + 8 * (y / 2)); };

        for (uint32_t i = 0; cur.pos < run.end && ok; i++) {
            const uint32_t row0 = cur.mt * C::kM + wm * 8 * RN;
            if (!begun) {
                begun = true;
                first = cur.tile;
                // This warp's queries, as the second operand: row g of each tile of eight.
#pragma unroll
                for (int t = 0; t < RN; t++) {
                    const uint32_t row = row0 + 8 * t + g;
                    const uint32_t tok = row / p.group, head = row - tok * p.group;
                    const bool have = row < p.rows;
                    const char* src = p.q.p + cur.b * p.q.b + (have ? tok * p.q.t + (uint64_t)(cur.h * p.group + head) * p.q.h : 0);
                    float top = 0.0f;
#pragma unroll
                    for (int kk = 0; kk < DP / 16; kk++)
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            const uint32_t d = kk * 16 + (FP8 ? 4 * l + 2 * y : 2 * l + 8 * y);
                            q[t][kk][y] = have && d < D ? *reinterpret_cast<const uint32_t*>(src + 2 * d) : 0;
                            if (!std::is_same<QT, T>::value) {
                                const QT* e = reinterpret_cast<const QT*>(&q[t][kk][y]);
                                top = fmaxf(top, fmaxf(fabsf(to_f32(e[0])), fabsf(to_f32(e[1]))));
                            }
                        }
                    float up = 1.0f;
                    if (!std::is_same<QT, T>::value) {
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        const RowScale scaled(top);
                        up = scaled.up;
#pragma unroll
                        for (int kk = 0; kk < DP / 16; kk++)
#pragma unroll
                            for (int y = 0; y < 2; y++) {
                                const QT* e = reinterpret_cast<const QT*>(&q[t][kk][y]);
                                q[t][kk][y] = pack2<__half>(to_f32(e[0]) * scaled.down, to_f32(e[1]) * scaled.down);
                            }
                    }
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        f[t][y] = p.scale * kLog2e * __shfl_sync(0xFFFFFFFFu, up, (2 * l + y) * 4);  // from a lane with that row
                        ref[t][y] = -INFINITY;
                        sum[t][y] = 0.0f;
                    }
                }
#pragma unroll
                for (int x = 0; x < DP / 16; x++)
#pragma unroll
                    for (int t = 0; t < RN; t++)
#pragma unroll
                        for (int y = 0; y < 4; y++) o[x][t][y] = 0.0f;
            }
            const uint32_t s = i % C::kStages;
            ok = warp_wait(full + 8 * s, (i / C::kStages) & 1);
            if (!ok) break;
            const uint32_t ks = smem_u32(smem + s * C::kStage), vs = ks + C::kTile * C::kRB;
            const uint32_t j0 = cur.tile * C::kTile + mykey;
            const bool masked = cur.tile * C::kTile + C::kTile > cur.span.old;

#pragma unroll
            for (int sub = 0; sub < C::kKeys / C::kSub; sub++) {
                const uint32_t key0 = mykey + sub * C::kSub;
                constexpr int kB = C::kSub / 16;             // blocks of 16 tokens
                constexpr int kChains = kB * RN == 1 ? 2 : 1;  // a lone accumulator would wait for itself at every step
                float sc[kChains][kB][RN][4];
#pragma unroll
                for (int h = 0; h < kChains; h++)
#pragma unroll
                    for (int x = 0; x < kB; x++)
#pragma unroll
                        for (int t = 0; t < RN; t++)
#pragma unroll
                            for (int y = 0; y < 4; y++) sc[h][x][t][y] = 0.0f;
#pragma unroll
                for (int x = 0; x < kB; x++) {
                    const uint32_t base = ks + row_chunk<C::kRB>(C::kTile, key0 + x * 16 + lane % 16, lane / 16);
                    if (!FP8) {
#pragma unroll
                        for (int kk = 0; kk < DP / 16; kk++) {
                            uint32_t a[4];
                            ldsm4(a, step_of(base, kk));
#pragma unroll
                            for (int t = 0; t < RN; t++) mma16816<T>(sc[kk % kChains][x][t], a, q[t][kk][0], q[t][kk][1]);
                        }
                    } else {
#pragma unroll
                        for (int kp = 0; kp < DP / 32; kp++) {
                            uint32_t r[4];
                            ldsm4(r, step_of(base, kp));
#pragma unroll
                            for (int y = 0; y < 2; y++) {
                                const uint32_t a[4] = {uzip::prmt(r[2 * y], 0, 0x1404), uzip::prmt(r[2 * y + 1], 0, 0x1404),
                                                       uzip::prmt(r[2 * y], 0, 0x3424), uzip::prmt(r[2 * y + 1], 0, 0x3424)};
#pragma unroll
                                for (int t = 0; t < RN; t++)
                                    mma16816<T>(sc[y % kChains][x][t], a, q[t][2 * kp + y][0], q[t][2 * kp + y][1]);
                            }
                        }
                    }
                }
                // Scores in units of log2: element y of a block is token g + 8 (y / 2) and row 2 l + y % 2.
                uint64_t seen[RN][2];
                if (masked)
#pragma unroll
                    for (int t = 0; t < RN; t++)
#pragma unroll
                        for (int y = 0; y < 2; y++)
                            seen[t][y] = seen_bits(p, cur.b, cur.span, row0 + 8 * t + 2 * l + y, j0 + sub * C::kSub);
                float most[RN][2];
                bool rise = false;
#pragma unroll
                for (int t = 0; t < RN; t++) {
                    most[t][0] = most[t][1] = -INFINITY;
#pragma unroll
                    for (int x = 0; x < kB; x++)
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            float v = sc[0][x][t][y];
                            if (kChains == 2) v += sc[kChains - 1][x][t][y];
                            v *= f[t][y & 1];
                            if (masked && !((seen[t][y & 1] >> (x * 16 + g + 8 * (y / 2))) & 1)) v = -INFINITY;
                            sc[0][x][t][y] = v;
                            most[t][y & 1] = fmaxf(most[t][y & 1], v);
                        }
                    rise |= most[t][0] > ref[t][0] + kSlack || most[t][1] > ref[t][1] + kSlack;
                }
                if (__any_sync(0xFFFFFFFFu, rise)) {
#pragma unroll
                    for (int t = 0; t < RN; t++) {
                        float fade[2];
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            float m = most[t][y];
                            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                            m = fmaxf(m, ref[t][y]);
                            fade[y] = ref[t][y] == -INFINITY ? 0.0f : exp2_fast(ref[t][y] - m);  // 0: nothing so far
                            ref[t][y] = m;
                            sum[t][y] *= fade[y];
                        }
#pragma unroll
                        for (int x = 0; x < DP / 16; x++)
#pragma unroll
                            for (int y = 0; y < 4; y++) o[x][t][y] *= fade[y & 1];
                    }
                }
                // Weights, rounded once to the products' 16 bits; their sum is of the unrounded ones. The matrix
                // instruction takes 16-bit operands, and the error is of the size of the output's own rounding. Outputs'
                // relative error against 64 bits, heads of 128 over 16,384 tokens: BF16 2.1e-3 (with 32-bit weights
                // 1.6e-3), FP16 2.6e-4 (2.0e-4).
                uint32_t w[kB][RN][2];
#pragma unroll
                for (int t = 0; t < RN; t++) {
                    const float r0 = ref[t][0] == -INFINITY ? 0.0f : ref[t][0] - kLift<T>;
                    const float r1 = ref[t][1] == -INFINITY ? 0.0f : ref[t][1] - kLift<T>;
#pragma unroll
                    for (int x = 0; x < kB; x++) {
                        const float e0 = exp2_fast(sc[0][x][t][0] - r0), e1 = exp2_fast(sc[0][x][t][1] - r1);
                        const float e2 = exp2_fast(sc[0][x][t][2] - r0), e3 = exp2_fast(sc[0][x][t][3] - r1);
                        sum[t][0] += e0 + e2;
                        sum[t][1] += e1 + e3;
                        w[x][t][0] = transpose8(pack2<T>(e0, e1));
                        w[x][t][1] = transpose8(pack2<T>(e2, e3));
                    }
                }
                // A value that a row does not see must not reach it through 0 * NaN: where the tile has new tokens,
                // non-finite values are taken out of the product and added below to the rows that see them.
                // (Rows past the last token may hold anything.)
                uint32_t odd = 0;
#pragma unroll
                for (int x = 0; x < kB; x++) {
                    uint32_t used[2] = {0, 0};  // halves of a pair of tokens 2 l, 2 l + 1 (and 8 on) that are in use
                    if (masked) {
                        const int32_t left = (int32_t)(cur.span.old + cur.span.fresh - (j0 + sub * C::kSub + x * 16)) - 2 * (int32_t)l;
                        for (int y = 0; y < 2; y++) used[y] = left - 8 * y >= 2 ? 0xFFFFFFFFu : left - 8 * y == 1 ? 0xFFFFu : 0;
                    }
                    if (!FP8) {
                        const uint32_t base = vs + row_chunk<C::kRB>(C::kTile, key0 + x * 16 + (lane / 16) * 8 + lane % 8, (lane / 8) % 2);
#pragma unroll
                        for (int dx = 0; dx < DP / 16; dx++) {
                            uint32_t a[4];
                            ldsm4_t(a, step_of(base, dx));
                            if (masked)
#pragma unroll
                                for (int y = 0; y < 4; y++) odd |= clean2<T>(a[y]) & used[y / 2];
#pragma unroll
                            for (int t = 0; t < RN; t++) mma16816<T>(o[dx][t], a, w[x][t][0], w[x][t][1]);
                        }
                    } else {
                        const uint32_t base = vs + row_chunk<C::kRB>(C::kTile, key0 + x * 16 + ((lane / 8) % 2) * 8 + lane % 8, lane / 16);
#pragma unroll
                        for (int dp = 0; dp < DP / 32; dp++) {
                            uint32_t r[4];
                            ldsm4_t(r, step_of(base, dp));
#pragma unroll
                            for (int y = 0; y < 2; y++) {
                                uint32_t a[4] = {uzip::prmt(r[2 * y], 0, 0x2404), uzip::prmt(r[2 * y], 0, 0x3414),
                                                 uzip::prmt(r[2 * y + 1], 0, 0x2404), uzip::prmt(r[2 * y + 1], 0, 0x3414)};
                                if (masked)
#pragma unroll
                                    for (int z = 0; z < 4; z++) odd |= clean2<T>(a[z]) & used[z / 2];
#pragma unroll
                                for (int t = 0; t < RN; t++) mma16816<T>(o[2 * dp + y][t], a, w[x][t][0], w[x][t][1]);
                            }
                        }
                    }
                }
                if (masked && __any_sync(0xFFFFFFFFu, odd != 0)) {
                    const uint32_t upto = cur.span.old + cur.span.fresh;
                    for (uint32_t k = 0; k < C::kSub; k++) {
                        const uint32_t j = j0 + sub * C::kSub + k;
                        if (j >= upto) break;
                        const Place pl = place_of(p.cache, cur.b, j);
                        if (pl.page < 0) continue;
                        const char* v = v_row(p.cache, pl, cur.h);
#pragma unroll
                        for (int x = 0; x < DP / 16; x++)
#pragma unroll
                            for (int y = 0; y < 4; y += 2) {
                                const uint32_t d = column(x, y);
                                if (d >= D) continue;
                                const float e = FP8 ? to_f32(reinterpret_cast<const E5M2*>(v)[d]) : to_f32(reinterpret_cast<const T*>(v)[d]);
                                if (isfinite(e)) continue;
#pragma unroll
                                for (int t = 0; t < RN; t++) {
                                    if ((seen[t][0] >> k) & 1) o[x][t][y] += e;
                                    if ((seen[t][1] >> k) & 1) o[x][t][y + 1] += e;
                                }
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(freed + 8 * s);

            const Unit done = cur;
            advance(p, cur, p.mtiles);
            const bool to_end = done.tile + 1 == done.tiles;
            if (!to_end && cur.pos < run.end) continue;
            // ---- end of the unit or of this CTA's run: merge the warps' token shares. A whole unit's rows are
            // finished, a part of one goes to the workspace.
            begun = false;
            const bool from_start = first == 0;
            float* const part = p.partial + ((uint64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * partial_floats(p);
#pragma unroll
            for (int t = 0; t < RN; t++) {
                float* mine = box + warp * 8 * C::kBoxRow;
#pragma unroll
                for (int x = 0; x < DP / 16; x++)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        float* at = mine + (2 * l + y) * C::kBoxRow + column(x, 0);
                        if (!FP8) {
                            at[0] = o[x][t][y];
                            at[8] = o[x][t][y + 2];
                        } else {
                            *reinterpret_cast<float2*>(at) = make_float2(o[x][t][y], o[x][t][y + 2]);
                        }
                    }
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    float v = sum[t][y];
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
                    if (g == 0) stat[warp * 8 + 2 * l + y] = make_float2(ref[t][y] == -INFINITY ? 0.0f : ref[t][y] - kLift<T>, v);
                }
                __syncwarp();
                if (lane == 0) bar_arrive(merge);
                ok = warp_wait(merge, merges++ & 1);
                if (!ok) break;
                // Four columns a thread, D / 4 threads a row.
                const uint32_t per = D / 4;
                for (uint32_t e = tid; e < WM * 8 * per; e += 256) {
                    const uint32_t r8 = e / per, d = (e - r8 * per) * 4, rm = r8 / 8, rn = r8 % 8;
                    const uint32_t r = rm * 8 * RN + 8 * t + rn, row = done.mt * C::kM + r;
                    if (row >= p.rows) continue;
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < C::kWN; k++) {
                        const float2 st = stat[(k * WM + rm) * 8 + rn];
                        if (st.y != 0.0f) top = fmaxf(top, st.x);
                    }
                    float all = 0.0f;
                    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < C::kWN; k++) {
                        const float2 st = stat[(k * WM + rm) * 8 + rn];
                        const float4 v = *reinterpret_cast<const float4*>(box + ((k * WM + rm) * 8 + rn) * C::kBoxRow + d);
                        if (st.y == 0.0f) continue;
                        const float e2 = exp2_fast(st.x - top);
                        all += st.y * e2;
                        acc.x += v.x * e2;
                        acc.y += v.y * e2;
                        acc.z += v.z * e2;
                        acc.w += v.w * e2;
                    }
                    const uint32_t tok = row / p.group, hq = done.h * p.group + (row - tok * p.group);
                    const bool none = tok >= done.span.fresh || all == 0.0f;
                    if (from_start && to_end) {
                        const float inv = none ? 0.0f : 1.0f / all;
                        *reinterpret_cast<uint2*>(p.out.p + done.b * p.out.b + tok * p.out.t + (uint64_t)hq * p.out.h + 2 * d) =
                            none ? make_uint2(0, 0)
                                 : make_uint2(pack2<QT>(acc.x * inv, acc.y * inv), pack2<QT>(acc.z * inv, acc.w * inv));
                        if (p.lse && d == 0)
                            p.lse[((uint64_t)done.b * p.tokens + tok) * p.q_heads + hq] = none ? -INFINITY : (top + log2f(all)) * kLn2;
                    } else {
                        *reinterpret_cast<float4*>(part + (uint64_t)r * DP + d) = acc;
                        if (d == 0) *reinterpret_cast<float2*>(part + (uint64_t)C::kM * DP + 2 * r) = make_float2(top, none ? 0.0f : all);
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(merge);
                ok = warp_wait(merge, merges++ & 1);
                if (!ok) break;
            }
        }
    }
    if (!ok && p.cache.status) *p.cache.status = UZIP_ERR_TIMEOUT;
}

template <typename QT, bool FP8, int DP, int RN, int WM>
int launch_attend_as(AttParams& p, int sms, cudaStream_t stream) {
    using C = AttCfg<QT, FP8, DP, RN, WM>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        UZIP_CUDA_TRY(cudaFuncSetAttribute(attend_kernel<QT, FP8, DP, RN, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem));
        // The shares that registers() hands out must be what the kernel is launched with, or it would wait forever.
        cudaFuncAttributes have;
        UZIP_CUDA_TRY(cudaFuncGetAttributes(&have, attend_kernel<QT, FP8, DP, RN, WM>));
        if (have.numRegs * kAttThreads < 4 * 32 * 72 + 8 * 32 * 216) return UZIP_ERR_CUDA;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    p.m = C::kM;
    p.mtiles = (p.rows + C::kM - 1) / C::kM;
    p.dp = DP;
    p.shift = C::kTile == 128 ? 7 : 6;
    p.unit_cost = 3;
    p.grid = std::min<uint32_t>((uint32_t)sms, kMaxAttGrid);
    attend_kernel<QT, FP8, DP, RN, WM><<<p.grid, kAttThreads, C::kSmem, stream>>>(p);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

// Rows a CTA takes at once: the fewest of 8, 16 and 32 that hold all (more rows of heads up to 128 go to the tensor
// cores instead, kManyRows); for larger heads of 16, 32 and 64, else 64.
template <typename QT, bool FP8, int DP>
int launch_attend_rows(AttParams& p, int sms, cudaStream_t s) {
    if constexpr (DP <= 128) {
        if (p.rows <= 8) return launch_attend_as<QT, FP8, DP, 1, 1>(p, sms, s);
        if (p.rows <= 16) return launch_attend_as<QT, FP8, DP, 2, 1>(p, sms, s);
        return launch_attend_as<QT, FP8, DP, 2, 2>(p, sms, s);
    } else {  // eight rows a warp: 16 would not leave registers for the output
        if (p.rows <= 16) return launch_attend_as<QT, FP8, DP, 1, 2>(p, sms, s);
        if (p.rows <= 32) return launch_attend_as<QT, FP8, DP, 1, 4>(p, sms, s);
        return launch_attend_as<QT, FP8, DP, 1, 8>(p, sms, s);
    }
}

template <typename QT, bool FP8>
int launch_attend(AttParams& p, int sms, cudaStream_t s) {
    if (p.cache.head_dim <= 64) return launch_attend_rows<QT, FP8, 64>(p, sms, s);
    if (p.cache.head_dim <= 128) return launch_attend_rows<QT, FP8, 128>(p, sms, s);
    return launch_attend_rows<QT, FP8, 256>(p, sms, s);
}

}  // namespace uzkv
