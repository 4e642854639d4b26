// kv_attend_many.cuh -- attention over a paged cache for many rows (large
// trees, many heads a KV head; head dimension up to 128) on the fifth-
// generation tensor cores.
//
// Bound: the tensor cores, 4 D flop a row and token. Two streams of work share
// a CTA: each has 128 rows of queries, two 128 x 64 score tiles and an output in
// tensor memory, a thread that issues its products, and a group of four warps
// in which a thread is a row, so the running reference and sum of its softmax
// are a thread's own. While the group turns one score tile into weights, the
// other one's product runs. A unit of more than 128 rows gives each stream 128
// of them, and both go through every tile of 128 cached tokens, half a tile at a
// time; one of up to 128 rows gives both streams the same rows, and they take
// the tiles in turn and are merged at its end.
//
//   S = Q K^T        Q and K tiles in shared memory, S in tensor memory
//   P = exp2(S - r)  by the stream's group; P, 16-bit, replaces S in tensor memory
//   O += P V         P from tensor memory, V from shared memory as it lies in the
//                    cache (the product's N, the head dimension, contiguous)
//
// Measured: 512 rows of 128 over two contexts of 65,536 tokens (252 GFLOP): 239 us, 1.05 PFLOP/s, 55 % of the measured
// cuBLAS rate; 85 rows of 64 over 12 E5M2 contexts of up to 5,001 tokens in pages of 48: 46 us, of 64: 40 us. One product
// thread for both streams and score tiles of 128 columns, one a stream, took 297 us: each stream's products then wait
// for its own softmax.
//
// Warps: 13 brings keys and values to a ring of operand tiles by bulk copies;
// 0-3 widen E5M2, which lands as bytes, take non-finite values out of tiles
// with new tokens, and do the copies where pages do not allow bulk ones; 4-7
// and 8-11 are the streams' groups, which also load their unit's queries and
// write its output; 12 and 14 issue the streams' products.
#pragma once

#include <algorithm>
#include <atomic>

#include "kv_tcgen05.cuh"

namespace uzkv {

constexpr int kManyThreads = 15 * 32;
constexpr uint32_t kManyTile = 128;

template <typename QT, bool FP8, int DP>
struct ManyCfg {
    using T = typename std::conditional<FP8, __half, QT>::type;
    static constexpr uint32_t kQTile = 128 * DP * 2;                 // queries of a stream
    static constexpr uint32_t kTileBytes = kManyTile * DP * 2;       // keys or values
    static constexpr uint32_t kRawBytes = kManyTile * DP;            // their E5M2 bytes
    static constexpr uint32_t kOther = 2560 + 512;                   // factors and statistics; barriers
    static constexpr uint32_t kRoom = 227 * 1024 - kOther - 2 * kQTile;
    static constexpr uint32_t kRaw = FP8 ? (DP == 64 ? 4 : 2) : 0;
    static constexpr uint32_t kFit = (kRoom - kRaw * kRawBytes) / kTileBytes;
    static constexpr uint32_t kTiles = kFit > 8 ? 8 : kFit;
    static constexpr uint32_t kRing = FP8 ? kRaw : kTiles;           // tiles on their way
    static constexpr uint32_t kSmem = kOther + 2 * kQTile + kTiles * kTileBytes + kRaw * kRawBytes;
    // A stream asks for its next tile's keys, two tiles on where the streams take turns, before it has given back the
    // values of its last: four operand tiles are the fewest that have room for that.
    static_assert(kTiles >= 4, "operand tiles");
};

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Descriptor of a tile whose contiguous dimension is the product's N: blocks of 64 elements `block` bytes apart,
// groups of 8 rows 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr, uint32_t block) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// One CTA's share of a unit. With up to 128 rows the streams take its tiles in turn, else both take each.
struct ManyPart {
    Unit u;
    uint32_t count, rows;  // tiles in this run; rows of the unit that exist
    bool both;             // more than 128 rows
    __device__ __forceinline__ ManyPart(const AttParams& p, const Unit& unit, uint64_t end) : u(unit) {
        count = (uint32_t)min((uint64_t)(u.tiles - u.tile), end - u.pos);
        rows = min(p.m, p.rows - u.mt * p.m);
        both = rows > 128;
    }
    // Half tiles of a stream, and the tile of one. The unit's last tile has one half where its tokens end in it.
    __device__ __forceinline__ uint32_t halves(uint32_t stream) const {
        const uint32_t tiles = both ? count : (count + 1 - stream) / 2;
        const bool last = u.tile + count == u.tiles && (both || (count - 1) % 2 == stream);
        return 2 * tiles - (last && (u.span.old + u.span.fresh - 1) % kManyTile < kManyTile / 2 ? 1 : 0);
    }
    __device__ __forceinline__ uint32_t tile_of(uint32_t stream, uint32_t half) const { return both ? half / 2 : half / 2 * 2 + stream; }
    __device__ __forceinline__ Unit next(const AttParams& p) const {
        Unit n = u;
        n.tile += count - 1;
        n.pos += count - 1;
        advance(p, n, p.mtiles);
        return n;
    }
};

template <typename QT, bool FP8, int DP, bool TMA>
__global__ void __launch_bounds__(kManyThreads, 1) attend_many_kernel(const __grid_constant__ AttParams p,
                                                                     const __grid_constant__ Maps maps) {
    using C = ManyCfg<QT, FP8, DP>;
    using T = typename C::T;
    extern __shared__ __align__(1024) char smem[];
    char* const qs = smem;
    char* const tiles = qs + 2 * C::kQTile;
    char* const raws = tiles + C::kTiles * C::kTileBytes;
    float* const factor = reinterpret_cast<float*>(raws + C::kRaw * C::kRawBytes);  // [256], or [128] of shared rows ...
    float2* const stat = reinterpret_cast<float2*>(factor + 128);  // ... and then [2][128]: each stream's reference and sum
    uint64_t* const bars = reinterpret_cast<uint64_t*>(factor + 640);
    uint32_t* const dirty = reinterpret_cast<uint32_t*>(bars + 48);  // [8]: a unit's tiles had non-finite values taken out
    uint32_t* const tmem_at = dirty + 8;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t D = p.cache.head_dim;
    const uint32_t full = smem_u32(bars), freed = full + 8 * 8, s_full = full + 16 * 8, p_full = full + 20 * 8,
                   o_ready = full + 24 * 8, q_full = full + 28 * 8, stat_full = full + 29 * 8, unit_done = full + 30 * 8,
                   landed = full + 32 * 8, raw_freed = full + 40 * 8;

    uzip::pdl_launch_dependents();
    if (tid == 0) {
        for (uint32_t i = 0; i < 8; i++) {
            bar_init(full + 8 * i, 4);       // the four warps that bring, widen or clean; bulk copies that need none of it
            bar_init(freed + 8 * i, 2);      // both streams
            bar_init(landed + 8 * i, TMA ? 1 : 128);  // copies for those warps
            bar_init(raw_freed + 8 * i, 4);  // E5M2 bytes: widened
            dirty[i] = 0;
        }
        for (uint32_t i = 0; i < 4; i++) {  // of a stream's two score tiles
            bar_init(s_full + 8 * i, 1);
            bar_init(p_full + 8 * i, 4);   // the four warps of the stream's group
            bar_init(o_ready + 8 * i, 1);  // the products with values of every other half tile
        }
        bar_init(q_full, 8);
        bar_init(stat_full, 8);
        bar_init(unit_done, 8);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) tc_alloc(smem_u32(tmem_at), 512);
    if (D < DP && (FP8 || !TMA)) {  // columns past the head dimension stay zero: no copy writes them
        for (uint32_t i = tid; i < C::kTiles * C::kTileBytes / 16; i += kManyThreads) reinterpret_cast<uint4*>(tiles)[i] = make_uint4(0, 0, 0, 0);
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    const Split split = split_of(p);
    const Run run = run_of(p, split, p.mtiles);
    Unit unit{};
    unit.pos = ~0ull;
    if (run.begin != run.end) unit = unit_at(p, split, run.begin, p.mtiles);
    bool ok = true;

    if (warp < 4) {
        // ---- copies: keys, then values of each tile; a warp takes 32 of its rows
        constexpr uint32_t kES = FP8 ? 1 : 2, kLanes = DP * kES / 16;  // a row's chunks
        constexpr uint32_t kRing = C::kRing;
        const uint32_t c = lane % kLanes, live = D * kES / 16;
        Unit ahead = unit;     // tile to copy next
        uint32_t copied = 0;   // operand tiles copied: even ones are keys
        Place at{0, 0};
        bool used = false;  // whether there is a token for this lane
        auto find = [&]() {
            Place pl{0, 0};
            const uint32_t j = ahead.tile * kManyTile + warp * 32 + lane;
            used = ahead.pos < run.end && j < ahead.span.old + ahead.span.fresh;
            if (used) pl = look_up(p.cache, ahead.b, j);
            return pl;
        };
        if (!TMA) at = find();
        auto copy = [&]() {  // the next operand tile's rows of this warp, to a slot that is free
            __syncwarp();
            const bool values = copied & 1;
            const Place now = used ? checked(p.cache, at) : Place{-1, 0};
            const char* row = now.page < 0 ? nullptr : values ? v_row(p.cache, now, ahead.h) : k_row(p.cache, now, ahead.h);
            const uint32_t s = copied % kRing;
            char* slot = (FP8 ? raws : tiles) + s * (FP8 ? C::kRawBytes : C::kTileBytes);
#pragma unroll 8
            for (uint32_t i = 0; i < kLanes; i++) {
                const uint32_t r = i * (32 / kLanes) + lane / kLanes;
                const char* src = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(row), r));
                const uint32_t R = warp * 32 + r;
                const uint32_t to = FP8 ? row_chunk<DP>(kManyTile, R, c) : swizzled(kManyTile, R, c);
                if (c < live) copy16(smem_u32(slot) + to, src ? src + c * 16 : p.cache.k, src != nullptr);
            }
            bar_arrive_copies(landed + 8 * s);
            copied++;
            if (values) {
                advance(p, ahead, p.mtiles);
                at = find();
            }
        };
        // As many copies as there is room for; waits for room only where nothing is left to hand on, because what frees
        // a slot may need the tiles that are already here.
        auto fill = [&](uint32_t sent) {
            while (ok && ahead.pos < run.end && copied < sent + kRing) {
                if (!FP8 && copied >= kRing) {
                    const uint32_t bar = freed + 8 * (copied % kRing), phase = (copied / kRing - 1) & 1;
                    if (copied > sent && !__all_sync(0xFFFFFFFFu, bar_test(bar, phase))) return;
                    ok = warp_wait(bar, phase);
                    if (!ok) return;
                }
                copy();
            }
        };
        Unit cur = unit;
        uint32_t sent = 0, index = 0, turns = 0;  // units so far; phases of `landed`, where only some tiles come through it
        while (cur.pos < run.end && ok) {
            const uint32_t j0 = cur.tile * kManyTile;
            for (uint32_t values = 0; values < 2 && ok; values++, sent++) {
                const bool clean = values && j0 + kManyTile > cur.span.old;
                if (!TMA) fill(sent);
                if (TMA && !FP8 && !clean) continue;
                const uint32_t at_slot = sent % kRing;
                if (ok) ok = warp_wait(landed + 8 * at_slot, FP8 || !TMA ? (sent / kRing) & 1 : (turns >> at_slot) & 1);
                turns ^= 1u << at_slot;
                if (!ok) break;
                char* const tile = tiles + (sent % C::kTiles) * C::kTileBytes;
                if (FP8) {
                    // Widen this warp's rows: 16 bytes to two chunks of eight FP16.
                    if (sent >= C::kTiles) ok = warp_wait(freed + 8 * (sent % C::kTiles), (sent / C::kTiles - 1) & 1);
                    if (!ok) break;
                    __syncwarp();
                    const char* raw = raws + (sent % kRing) * C::kRawBytes;
                    constexpr uint32_t kBatch = kLanes < 8 ? kLanes : 8;  // all read before the first is written
                    if (c < live)
#pragma unroll
                        for (uint32_t x0 = 0; x0 < kLanes; x0 += kBatch) {
                            uint4 v[kBatch];
#pragma unroll
                            for (uint32_t x = 0; x < kBatch; x++)
                                v[x] = *reinterpret_cast<const uint4*>(raw + row_chunk<DP>(kManyTile, warp * 32 + (x0 + x) * (32 / kLanes) + lane / kLanes, c));
#pragma unroll
                            for (uint32_t x = 0; x < kBatch; x++) {
                                const uint32_t R = warp * 32 + (x0 + x) * (32 / kLanes) + lane / kLanes;
                                *reinterpret_cast<uint4*>(tile + swizzled(kManyTile, R, 2 * c)) = widen(v[x].x, v[x].y);
                                *reinterpret_cast<uint4*>(tile + swizzled(kManyTile, R, 2 * c + 1)) = widen(v[x].z, v[x].w);
                            }
                        }
                }
                if (clean) {
                    // A value that a row does not see must not reach it through 0 * NaN: non-finite values of a tile
                    // with new tokens leave it here, and the unit's end adds them to the rows that see them. Rows past
                    // the last token, which a bulk copy may have brought, become zeros. Each thread looks at the
                    // chunks of its warp's rows that it wrote, or would have.
                    bool bad = false;
                    const uint32_t end = cur.span.old + cur.span.fresh;
                    if (c < live)
                        for (uint32_t x = 0; x < kLanes; x++) {
                            const uint32_t R = warp * 32 + x * (32 / kLanes) + lane / kLanes;
                            for (uint32_t half = 0; half < (FP8 ? 2 : 1); half++) {
                                uint4* at16 = reinterpret_cast<uint4*>(tile + swizzled(kManyTile, R, FP8 ? 2 * c + half : c));
                                if (j0 + R >= end) {
                                    *at16 = make_uint4(0, 0, 0, 0);
                                    continue;
                                }
                                uint4 v = *at16;
                                if (clean2<T>(v.x) | clean2<T>(v.y) | clean2<T>(v.z) | clean2<T>(v.w)) {
                                    *at16 = v;
                                    bad = true;
                                }
                            }
                        }
                    if (bad) *reinterpret_cast<volatile uint32_t*>(dirty + index % 8) = 1;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(full + 8 * (sent % C::kTiles));
                    if (TMA && FP8) bar_arrive(raw_freed + 8 * (sent % kRing));
                }
            }
            const bool to_end = cur.tile + 1 == cur.tiles;
            advance(p, cur, p.mtiles);
            if (to_end) index++;
        }
        if (!TMA) asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 13) {
        // ---- bulk copies: keys, then values of each tile
        if (TMA) {
            using Feed = TmaFeed<kManyTile, FP8 ? DP : DP * 2>;
            char* const ring = FP8 ? raws : tiles;
            const uint32_t again = FP8 ? raw_freed : freed;
            Feed feed;
            feed.find(p, maps, unit, unit.pos < run.end);
            uint32_t n = 0;  // operand tiles
            while (unit.pos < run.end && ok) {
                const Feed now = feed;
                const uint32_t h = unit.h;
                const bool masked = (unit.tile + 1) * kManyTile > unit.span.old;
                advance(p, unit, p.mtiles);
                feed.find(p, maps, unit, unit.pos < run.end);
                for (uint32_t values = 0; values < 2 && ok; values++, n++) {
                    const uint32_t s = n % C::kRing;
                    if (n >= C::kRing) ok = warp_wait(again + 8 * s, (n / C::kRing - 1) & 1);
                    if (!ok) break;
                    const bool by = FP8 || (values && masked);  // the warps that widen or clean come first
                    const uint32_t done = (by ? landed : full) + 8 * s;
                    if (lane == 0) {
                        bar_expect(done, now.bytes(maps));
                        if (!by) bar_arrive(done, 3);
                    }
                    __syncwarp();
                    now.copy(p, maps, values ? &maps.v : &maps.k, h, smem_u32(ring + s * (FP8 ? C::kRawBytes : C::kTileBytes)), done);
                }
            }
            const uint32_t last = FP8 ? landed : full;
            for (uint32_t k = n > C::kRing ? n - C::kRing : 0; k < n; k++)  // no copy outlives the CTA
                ok &= warp_wait(last + 8 * (k % C::kRing), (k / C::kRing) & 1);
        }
    } else if (warp == 12 || warp == 14) {
        // ---- a stream's products, by one lane
        if (lane == 0) {
            const uint32_t x = warp == 12 ? 0 : 1;
            const uint32_t n = (D + 15) / 16 * 16;  // columns of the output
            const uint32_t iqk = mma_desc<T>(128, 64), ipv = mma_desc<T>(128, n) | 1u << 16;  // V: N contiguous
            // Descriptors once; offsets add to their low bits.
            const uint64_t q0 = tile_desc(smem_u32(qs)), k0 = tile_desc(smem_u32(tiles)), v0 = rows_desc(smem_u32(tiles), kManyTile * 128);
            uint32_t base = 0, index = 0, turns = 0;  // operand tiles of earlier units; units; phases of the two p_full
            while (unit.pos < run.end && ok) {
                const ManyPart part(p, unit, run.end);
                const uint32_t halves = part.halves(x);
                const uint64_t q = q0 + (part.both ? x * (C::kQTile >> 4) : 0);
                auto wait_full = [&](uint32_t t) { return bar_wait(full + 8 * (t % C::kTiles), (t / C::kTiles) & 1); };
                auto pass = [&](uint32_t tile) {  // a tile of the other stream's: give it back as soon as it is there
                    for (uint32_t t = base + 2 * tile; ok && t < base + 2 * tile + 2; t++) {
                        ok = wait_full(t);
                        if (ok) bar_arrive(freed + 8 * (t % C::kTiles));
                    }
                };
                auto score = [&](uint32_t h) {
                    const uint32_t tile = part.tile_of(x, h), t = base + 2 * tile, s = t % C::kTiles;
                    if (!(h & 1)) {
                        if (!part.both && tile) pass(tile - 1);
                        if (ok) ok = wait_full(t);
                        if (!ok) return;
                    }
                    tc_fence_after();
                    const uint64_t k = k0 + s * (C::kTileBytes >> 4) + (h & 1) * (64 * 128 >> 4);
                    tc_mma_steps<DP / 16>(tmem + x * 256 + (h & 1) * 64, q, 128 * 128 >> 4, k, kManyTile * 128 >> 4, iqk);
                    tc_commit(s_full + 8 * (2 * x + (h & 1)));
                    if ((h & 1) || h + 1 == halves) tc_commit(freed + 8 * s);
                };
                ok = bar_wait(q_full, index & 1);
                if (ok && halves) score(0);
                if (ok && halves > 1) score(1);
                for (uint32_t h = 0; h < halves && ok; h++) {
                    const uint32_t t = base + 2 * part.tile_of(x, h) + 1, s = t % C::kTiles, b = h & 1;
                    if (!b) ok = wait_full(t);
                    if (ok) ok = bar_wait(p_full + 8 * (2 * x + b), (turns >> b) & 1);
                    turns ^= 1u << b;
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = v0 + s * (C::kTileBytes >> 4) + b * (64 * 128 >> 4);
#pragma unroll
                    for (uint32_t i = 0; i < 4; i++)
                        tc_mma_ts(tmem + x * 256 + 128, tmem + x * 256 + b * 64 + i * 8, v + i * (2048 >> 4), ipv, h != 0 || i != 0);
                    tc_commit(o_ready + 8 * (2 * x + b));
                    if (b || h + 1 == halves) tc_commit(freed + 8 * s);
                    if (h + 2 < halves) score(h + 2);
                }
                if (!part.both) {  // tiles of the other stream's after this one's last
                    const uint32_t mine = (halves + 1) / 2, next = mine ? 2 * (mine - 1) + x + 1 : 0;
                    for (uint32_t tile = next; tile < part.count && ok; tile++) pass(tile);
                }
                base += 2 * part.count;
                index++;
                unit = part.next(p);
            }
        }
        __syncwarp();
    } else {
        // ---- a stream's softmax, queries and output: thread `row` of 128
        const uint32_t x = warp < 8 ? 0 : 1, row = (warp % 4) * 32 + lane;
        const uint32_t lanes = warp % 4 * 32 << 16, st = tmem + x * 256 + lanes, ot = st + 128;
        uint32_t index = 0, turns = 0;          // units; phases of the two s_full
        // Products with values of this stream in earlier units, by half. When a half tile's scores are there, the
        // products of the last one but one are complete, so of a barrier's phases at most one is open.
        uint32_t products[2] = {0, 0};
        while (unit.pos < run.end && ok) {
            const ManyPart part(p, unit, run.end);
            const Unit& u = part.u;
            const uint32_t row0 = u.mt * p.m;
            if (part.both)
                load_queries<QT, T, DP, 128>(
                    p, tid % 128, u.b, u.h, row0 + x * 128, 128,
                    [&](uint32_t r, uint32_t ch) { return reinterpret_cast<uint4*>(qs + x * C::kQTile + swizzled(128, r, ch)); },
                    factor + x * 128);
            else  // half of the shared rows each
                load_queries<QT, T, DP, 128>(
                    p, tid % 128, u.b, u.h, row0 + x * 64, 64,
                    [&](uint32_t r, uint32_t ch) { return reinterpret_cast<uint4*>(qs + swizzled(128, x * 64 + r, ch)); },
                    factor + x * 64);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(q_full);
            ok = warp_wait(q_full, index & 1);  // factors of the other warps too
            if (!ok) break;
            const uint32_t mine = part.both ? x * 128 + row : row;  // row of the unit
            float f = factor[mine];
            if (f == 0.0f) f = 1.17549435e-38f;  // the smallest normal number: 0 * -inf would be no number
            float ref = -INFINITY, sum = 0.0f;
            const uint32_t halves = part.halves(x);
            for (uint32_t h = 0; h < halves; h++) {
                const uint32_t b = h & 1, at = st + b * 64, j0 = (u.tile + part.tile_of(x, h)) * kManyTile + b * 64;
                ok = warp_wait(s_full + 8 * (2 * x + b), (turns >> b) & 1);
                turns ^= 1u << b;
                if (!ok) break;
                tc_fence_after();
                uint32_t v[64];
                tc_ld32(v, at);
                tc_ld32(v + 32, at + 32);
                uint64_t seen = ~0ull;
                if (j0 + 64 > u.span.old) seen = seen_bits(p, u.b, u.span, row0 + mine, j0);
                tc_wait_ld();
                if (j0 + 64 > u.span.old) {
#pragma unroll
                    for (int i = 0; i < 64; i++)
                        if (!((uint32_t)(seen >> (i & 32)) >> (i & 31) & 1)) v[i] = 0xFF800000u;  // -inf
                }
                float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                    most[i / 2 % 4] = fmaxf(most[i / 2 % 4], fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                float high = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                high *= f;  // f is positive
                if (__any_sync(0xFFFFFFFFu, high > ref + kSlack)) {  // the reference may trail by kSlack
                    const float now = fmaxf(ref, high);
                    const float fade = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);  // 0: nothing so far
                    ref = now;
                    sum *= fade;
                    if (h > 0) {  // the last product with values may still run
                        ok = warp_wait(o_ready + 8 * (2 * x + 1 - b), ((b ? products[0] : products[1]) + (h - 1) / 2) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        for (uint32_t c = 0; c < D; c += 16) {
                            float z[16];
                            tc_ld16(z, ot + c);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; i++) z[i] *= fade;
                            tc_st16(ot + c, reinterpret_cast<const uint32_t*>(z));
                        }
                    }
                }
                // Weights take the scores' place, 32 columns for 64: rounded once to the 16 bits that the product takes,
                // their sum of the unrounded ones (errors as in the small-row kernel: BF16 2.2e-3 for 1.7e-3).
                const float r = ref == -INFINITY ? 0.0f : ref - kLift<T>;
                const uint64_t f2 = pair(f, f), r2 = pair(-r, -r);
                uint64_t add[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const uint32_t *y = v + 32 * c + i;
                        float2 a = unpair(fma2(pair(__uint_as_float(y[0]), __uint_as_float(y[1])), f2, r2));
                        a.x = exp2_fast(a.x);
                        a.y = exp2_fast(a.y);
                        add[i / 2 & 1] = add2(add[i / 2 & 1], pair(a.x, a.y));
                        w[i / 2] = pack2<T>(a.x, a.y);
                    }
                    tc_st16(at + 16 * c, w);
                }
                const float2 total = unpair(add2(add[0], add[1]));
                sum += total.x + total.y;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full + 8 * (2 * x + b));
            }
            if (!ok) break;
            // ---- output
            if (halves) {
                const uint32_t b = (halves - 1) & 1;
                ok = warp_wait(o_ready + 8 * (2 * x + b), ((b ? products[1] : products[0]) + (halves - 1) / 2) & 1);
            }
            products[0] += (halves + 1) / 2;
            products[1] += halves / 2;
            if (!ok) break;
            tc_fence_after();
            float mref = ref == -INFINITY ? 0.0f : ref - kLift<T>;
            // Streams that took the tiles of the same rows in turn: each merges half of the columns.
            float2 other = make_float2(0.0f, 0.0f);
            if (!part.both) stat[x * 128 + row] = make_float2(mref, sum);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(stat_full);
            ok = warp_wait(stat_full, index & 1);  // the other stream's output is complete too
            if (!ok) break;
            tc_fence_after();
            const bool odd = *reinterpret_cast<volatile uint32_t*>(dirty + index % 8) != 0;
            float keep = 1.0f, give = 0.0f;
            if (!part.both) {
                other = stat[(1 - x) * 128 + row];
                const float top = sum == 0.0f ? other.x : other.y == 0.0f ? mref : fmaxf(mref, other.x);
                keep = sum == 0.0f ? 0.0f : exp2_fast(mref - top);
                give = other.y == 0.0f ? 0.0f : exp2_fast(other.x - top);
                sum = (sum == 0.0f ? 0.0f : sum * keep) + (other.y == 0.0f ? 0.0f : other.y * give);
                mref = top;
            }
            const uint32_t grow = row0 + mine, tok = grow / p.group, hq = u.h * p.group + (grow - tok * p.group);
            const bool exists = grow < p.rows, none = !exists || tok >= u.span.fresh || sum == 0.0f;
            const bool from_start = u.tile == 0, to_end = u.tile + part.count == u.tiles;
            const float inv = none ? 0.0f : 1.0f / sum;
            float* const dst = p.partial + ((uint64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * partial_floats(p);
            char* const out = p.out.p + u.b * p.out.b + tok * p.out.t + (uint64_t)hq * p.out.h;
            const uint32_t ot0 = tmem + 128 + lanes;
            for (uint32_t c = 0; c < D; c += 32) {
                if (!part.both && (c / 32 & 1) != x) continue;
                uint32_t v[32];
                __syncwarp();
                if (part.both) {
                    tc_ld32(v, ot + c);
                    tc_wait_ld();
                } else {
                    uint32_t o2[32];
                    tc_ld32(v, (x ? ot0 + 256 : ot0) + c);
                    tc_ld32(o2, (x ? ot0 : ot0 + 256) + c);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i++) {  // a stream without weight may have no output at all
                        const float a = keep == 0.0f ? 0.0f : __uint_as_float(v[i]) * keep;
                        const float b = give == 0.0f ? 0.0f : __uint_as_float(o2[i]) * give;
                        v[i] = __float_as_uint(a + b);
                    }
                }
                if (odd && exists) {
                    const uint32_t upto = min((u.tile + part.count) * kManyTile, u.span.old + u.span.fresh);
                    const uint32_t from = max(u.tile * kManyTile, u.span.old / kManyTile * kManyTile);
                    for (uint32_t j = from; j < upto; j++) {
                        if (!(seen_bits(p, u.b, u.span, grow, j) & 1)) continue;
                        const Place pl = place_of(p.cache, u.b, j);
                        if (pl.page < 0) continue;
                        const char* vr = v_row(p.cache, pl, u.h);
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            if (c + i >= D) continue;
                            const float e = FP8 ? to_f32(reinterpret_cast<const E5M2*>(vr)[c + i]) : to_f32(reinterpret_cast<const T*>(vr)[c + i]);
                            if (!isfinite(e)) v[i] = __float_as_uint(__uint_as_float(v[i]) + e);
                        }
                    }
                }
                if (!exists) {
                } else if (from_start && to_end) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (c + i >= D) continue;
                        uint4 y = make_uint4(0, 0, 0, 0);
                        if (!none) {
                            uint32_t* z = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                z[k] = pack2<QT>(__uint_as_float(v[i + 2 * k]) * inv, __uint_as_float(v[i + 2 * k + 1]) * inv);
                        }
                        *reinterpret_cast<uint4*>(out + 2 * (c + i)) = y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (c + i < D)
                            *reinterpret_cast<uint4*>(dst + (uint64_t)mine * DP + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (exists && (part.both || x == 0)) {
                if (from_start && to_end) {
                    if (p.lse) p.lse[((uint64_t)u.b * p.tokens + tok) * p.q_heads + hq] = none ? -INFINITY : (mref + log2f(sum)) * kLn2;
                } else {
                    *reinterpret_cast<float2*>(dst + (uint64_t)p.m * DP + 2 * mine) = make_float2(mref, none ? 0.0f : sum);
                }
            }
            // All reads of the unit's accumulators, statistics and flag are over before the next unit's queries are announced.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(unit_done);
            ok = warp_wait(unit_done, index & 1);
            if (!ok) break;
            if (odd && x == 0 && row == 0) *reinterpret_cast<volatile uint32_t*>(dirty + index % 8) = 0;
            index++;
            unit = part.next(p);
        }
    }
    if (!ok && p.cache.status) *p.cache.status = UZIP_ERR_TIMEOUT;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tc_free(tmem, 512);
}

template <typename QT, bool FP8, int DP, bool TMA>
int launch_many_by(AttParams& p, const Maps& maps, cudaStream_t stream) {
    using C = ManyCfg<QT, FP8, DP>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device whose limit is raised
    int dev = 0;
    UZIP_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        UZIP_CUDA_TRY(cudaFuncSetAttribute(attend_many_kernel<QT, FP8, DP, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem));
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    attend_many_kernel<QT, FP8, DP, TMA><<<p.grid, kManyThreads, C::kSmem, stream>>>(p, maps);
    UZIP_CUDA_TRY(cudaGetLastError());
    return UZIP_OK;
}

template <typename QT, bool FP8, int DP>
int launch_many_as(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t stream) {
    p.m = p.rows <= 128 ? 128 : 256;
    p.mtiles = (p.rows + p.m - 1) / p.m;
    p.dp = DP;
    p.shift = 7;
    static_assert(kManyTile == 1u << 7, "tile");
    p.unit_cost = 5;
    p.grid = std::min<uint32_t>((uint32_t)sms, kMaxAttGrid);
    Maps maps{};
    if (maps_of(p, c, kManyTile, 2048, &maps)) return launch_many_by<QT, FP8, DP, true>(p, maps, stream);
    return launch_many_by<QT, FP8, DP, false>(p, maps, stream);
}

template <typename QT, bool FP8>
int launch_many(AttParams& p, const uzkv_cache_t* c, int sms, cudaStream_t s) {
    return p.cache.head_dim <= 64 ? launch_many_as<QT, FP8, 64>(p, c, sms, s) : launch_many_as<QT, FP8, 128>(p, c, sms, s);
}

}  // namespace uzkv
