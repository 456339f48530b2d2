// paged_attn.cuh -- what the paged-attention kernels share: the division of the work among
// the CTAs, the scheduler warp that hands it out, and the TMA producer warp.
//
// A unit is the rows of one KV head's query heads for up to `tpu` consecutive new tokens of
// one request (G query heads per KV head, rows token-major).
//   all keys         the (unit, key tile) pairs of all units form one line that is cut into
//                    one equal piece per CTA (one CTA per SM), whatever the lengths are; a
//                    unit cut by a piece's end leaves fp32 partial results that
//                    k_paged_merge joins in a fixed order.  Where whole units, dealt out
//                    evenly, take no longer than equal pieces and their merge
//                    (kMergeCost), nothing is cut.
//   selected blocks  a unit is one token and walks the list of its valid blocks.  Units go
//                    round the CTAs, all tokens of a KV head before the next head, so that
//                    the tokens of a chunk find the head's blocks in L2; the units that do
//                    not fill a last round form a line as above, by the same rule.
//
// Keys that no row of a unit may see are never read into a product: their pages are not
// loaded, and the issuers leave out the 16-key steps of P V without a visible key and
// clear the dead rows of V in the others (0 times infinity is not 0).
#pragma once

#include <math_constants.h>

#include "paged.h"

namespace nsa {

constexpr int kTileKeys = 128;
constexpr int kRegion = kTileKeys * 128;     // bytes of 128 rows x 64 columns
// A K or V tile in shared memory: groups of 8 keys, in each the 64-column halves one after the
// other (8 rows of 128 bytes, 128-byte swizzle).  A box of whole rows is then contiguous, so that
// a page takes one TMA load; a box costs the TMA unit about 50 cycles next to its bytes (pages of
// 16, a box per half: 18 bytes a cycle and SM; pages of 64: 28).
template <int D>
struct Tile {
    static constexpr uint32_t kGroup = D * 16;                 // bytes of 8 keys
    static constexpr uint32_t kGroupU = kGroup >> 4, kHalfU = 1024 >> 4;   // descriptor units
    // the upper word of the descriptors (those of Q and P: kSw128Sbo1024DescHi)
    static constexpr uint32_t kDescHi = (kGroup >> 4) | 1u << 14 | 2u << 29;
};
constexpr int kUnitCost = 1;                 // a unit's prologue and epilogue, in key tiles
constexpr int kMergeCost = 6;                // writing and joining partial results, in key tiles
constexpr float kLazy = 8.f;

// A CTA's share of a unit: key tiles [p0, p1) of its nt.
struct Piece {
    int tok0, ntok, g, r;
    int pos0;           // position of the first token
    int lo, hi;         // keys that some row sees lie in [lo, hi]
    int tile0;          // all keys: the first key tile's number
    int nb;             // selected blocks: entries of the list
    int p0, p1, nt;
    int slot;           // partial slot, or -1: the piece is the whole unit
    int more;           // 0: no piece, the CTA is done
};

constexpr int kRing = 8;

struct Params {
    PagedAttnArgs a;
    int tpt;            // tokens per tile of query rows
    int tpu;            // tokens per unit
    int box_rows;       // keys of one K / V box
    int page_groups;    // > 0: places of a page in the maps' dimension of 8-key groups; 0: the maps
                        // have dimensions of keys and pages, and boxes of 8 keys
    int cost_sel;       // selected blocks: places of a unit on the line
    bool whole_sel;     // and whether the last round's units stay whole
    float* part_o;      // [pieces][NQ * 128][D]
    float2* part_ml;    // [pieces][NQ * 128] (m, l)
    int4* desc;         // [grid] unit left open by CTA c: (token, ntok, g, last CTA) or last = -1
};

// (whole rows: the coordinates of the columns are 0)
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int c1, int c3,
                                              int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c3), "r"(c4)
        : "memory");
}
// mma_ss_e and mma_ts_e with the upper words of the operands' descriptors
__device__ __forceinline__ void mma_ss_hi(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t accumulate, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "mov.b64 da, {%1, %6};\n\t"
        "mov.b64 db, {%2, %7};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(a_hi), "r"(b_hi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_hi(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t idesc, uint32_t accumulate, uint32_t elected) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "mov.b64 db, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(b_hi)
        : "memory");
}
// Clears rows [from, to) of a tile, by one warp.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int lane) {
    for (int r = from; r < to; ++r)
        if (lane < D / 8)
            *reinterpret_cast<uint4*>(tile + (r >> 3) * Tile<D>::kGroup + (lane >> 3) * 1024 + (r & 7) * 128 +
                                      (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
}
// 16 consecutive fp32 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld16_sync(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "{\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st16_sync(uint32_t taddr, const float* v) {
    const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
    asm volatile(
        "{\n\t"
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
        "tcgen05.wait::st.sync.aligned;\n\t}"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Request r: rows [a, a + n) of q, kv keys, all inside their buffers whatever the arrays say.
struct Req { int a, n, kv; };
__device__ __forceinline__ Req request(const PagedAttnArgs& p, int r) {
    Req q;
    q.a = min(max(p.cu[r], 0), p.T);
    q.n = min(max(p.cu[r + 1], q.a), p.T) - q.a;
    q.kv = min(max(p.kv_lens[r], 0), p.table_width * p.ps);
    return q;
}
__device__ __forceinline__ bool request_ok(const PagedAttnArgs& p, int r) {
    const int a = p.cu[r], b = p.cu[r + 1], kv = p.kv_lens[r];
    return a >= 0 && b >= a && b <= p.T && kv >= 0 && kv <= p.table_width * p.ps;
}

// Visible keys of tokens [t, t + ntok) of a request, as [lo, hi]; key tiles touched.
__device__ __forceinline__ void unit_keys(const Req& q, int t, int ntok, int swin, int* pos0, int* lo,
                                          int* hi, int* nt) {
    *pos0 = q.kv - q.n + t;
    *hi = *pos0 + ntok - 1;                    // < kv
    *lo = swin > 0 ? max(0, *pos0 - swin + 1) : 0;
    *nt = *hi < 0 ? 0 : *hi / kTileKeys - *lo / kTileKeys + 1;
}

// A line of `total` places cut into `pieces` equal parts: the part that holds place x.
__device__ __forceinline__ long long quotient(long long a, long long b) {   // of a, b >= 0
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int owner_of(long long x, long long total, long long pieces) {
    return (int)quotient((x + 1) * pieces - 1, total);
}

// A unit's piece [u0, u1) of its nt + kUnitCost places (the last ones hold no key tile) as
// key tiles.  False if it holds none, but for a unit without a key tile (nt = 0): write_empty().
__device__ __forceinline__ bool piece_tiles(long long u0, long long u1, int cta, Piece& k) {
    k.p0 = (int)min(u0, (long long)k.nt);
    k.p1 = (int)min(u1, (long long)k.nt);
    k.slot = k.p0 == 0 && k.p1 == k.nt ? -1 : 2 * cta + (k.p0 == 0 ? 1 : 0);
    k.more = 1;
    return k.p0 < k.p1 || (k.nt == 0 && u0 == 0);
}

// All keys: a CTA's piece [x, x1) of the line of (KV head, request, tile of tokens, key
// tile).  Run by one warp.  start(): every CTA sums the costs of all requests by itself,
// lanes over requests (over the tiles of tokens of a long one), from the lengths alone.
struct WalkAll {
    long long x, x1, u0, total, pieces;
    long long unit_at;    // place of the piece's unit on the line
    int head, r, qt;
    bool whole;           // a unit is one place: nothing is cut
    __device__ __forceinline__ int tile_cost(const PagedAttnArgs& p, const Req& q, int i, int tpu) const {
        if (whole) return 1;
        int pos0, lo, hi, nt;
        unit_keys(q, i * tpu, min(tpu, q.n - i * tpu), p.swin, &pos0, &lo, &hi, &nt);
        return nt + kUnitCost;
    }
    __device__ __forceinline__ static long long scan(long long v, int lane) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    }
    // every lane's own request
    __device__ __forceinline__ long long cost(const PagedAttnArgs& p, const Req& q, int tpu, int lane) const {
        const int tiles = (q.n + tpu - 1) / tpu;
        long long c = 0;
        if (tiles <= 2)
            for (int i = 0; i < tiles; ++i) c += tile_cost(p, q, i, tpu);
        for (unsigned many = __ballot_sync(0xffffffffu, tiles > 2); many; many &= many - 1) {
            const int src = __ffs(many) - 1;
            const Req h{0, __shfl_sync(0xffffffffu, q.n, src), __shfl_sync(0xffffffffu, q.kv, src)};
            long long sum = 0;
            for (int i = lane; i < (h.n + tpu - 1) / tpu; i += 32) sum += tile_cost(p, h, i, tpu);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == src) c = sum;
        }
        return c;
    }
    // false: the lengths are not sound.  Requests that overlap get no work: the line's sums hold
    // for total_tokens tokens, not for more.
    __device__ __forceinline__ bool start(const Params& P, int tpu, int cta, int grid, int lane) {
        const PagedAttnArgs& p = P.a;
        const int per = (p.R + 31) / 32;
        long long mine = 0;
        int count = 0, tokens = 0;
        int most = 0;                       // costs of the most expensive unit
        bool good = true;
        whole = false;
        x = x1 = u0 = 0;
        auto load = [&](int i, int end) {
            Req q{0, 0, 0};
            if (i < end) q = request(p, i);
            return q;
        };
        for (int s = 0; s < per; ++s) {
            const int i = lane * per + s;
            const Req q = load(i, p.R);
            if (i < p.R) good &= request_ok(p, i);
            tokens += __reduce_add_sync(0xffffffffu, q.n);
            if (tokens > p.T) return false;
            mine += cost(p, q, tpu, lane);
            const int last = (q.n + tpu - 1) / tpu - 1;
            count += last + 1;
            if (last >= 0)                  // (the last tile of tokens sees as many keys as any)
                most = max(most, max(tile_cost(p, q, last, tpu), tile_cost(p, q, max(last - 1, 0), tpu)));
        }
        long long inc = scan(mine, lane);
        long long all = __shfl_sync(0xffffffffu, inc, 31);
        // (units of one KV head: at most total_tokens)
        const long long units = (long long)__reduce_add_sync(0xffffffffu, count) * p.hkv;
        most = __reduce_max_sync(0xffffffffu, most);
        whole = quotient(units + grid - 1, grid) * most <= quotient(all * p.hkv + grid - 1, grid) + kMergeCost;
        if (whole) {
            mine = count;
            inc = scan(mine, lane);
            all = __shfl_sync(0xffffffffu, inc, 31);
        }
        total = all * p.hkv;
        pieces = min((long long)grid, total);
        head = r = qt = 0;
        good = __all_sync(0xffffffffu, good);
        if (cta >= pieces) return good;
        x = quotient(cta * total, pieces);
        x1 = quotient((cta + 1) * total, pieces);
        head = (int)quotient(x, all);
        long long off = x - head * all;      // in the head's part of the line
        const unsigned holds = __ballot_sync(0xffffffffu, off < inc);
        const int owner = __ffs(holds) - 1;
        off -= __shfl_sync(0xffffffffu, inc - mine, owner);
        r = owner * per;
        if (per > 1) {                       // the request, among the owner's
            const int end = min(p.R, (owner + 1) * per);
            for (int base = r; base < end; base += 32) {
                const long long c = cost(p, load(base + lane, end), tpu, lane), ci = scan(c, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, off < ci);
                if (hit) {
                    const int l = __ffs(hit) - 1;
                    off -= __shfl_sync(0xffffffffu, ci - c, l);
                    r = base + l;
                    break;
                }
                off -= __shfl_sync(0xffffffffu, ci, 31);
            }
        }
        const Req q = request(p, r);
        for (int base = 0; q.n > tpu && base * tpu < q.n; base += 32) {   // its tile of tokens
            const int i = base + lane;
            const long long c = i * tpu < q.n ? tile_cost(p, q, i, tpu) : 0, ci = scan(c, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, off < ci);
            if (hit) {
                const int l = __ffs(hit) - 1;
                off -= __shfl_sync(0xffffffffu, ci - c, l);
                qt = base + l;
                break;
            }
            off -= __shfl_sync(0xffffffffu, ci, 31);
        }
        u0 = off;
        return good;
    }
    __device__ __forceinline__ bool next(const Params& P, int tpu, int cta, Piece& k) {
        const PagedAttnArgs& p = P.a;
        while (x < x1) {
            Req q = request(p, r);
            while ((long long)qt * tpu >= q.n) {
                qt = 0;
                if (++r == p.R) {
                    r = 0;
                    if (++head >= p.hkv) return false;   // (lengths that changed under the call)
                }
                q = request(p, r);
            }
            const int t = qt * tpu;
            k.ntok = min(tpu, q.n - t);
            k.tok0 = q.a + t;
            k.g = head;
            k.r = r;
            unit_keys(q, t, k.ntok, p.swin, &k.pos0, &k.lo, &k.hi, &k.nt);
            k.tile0 = k.lo / kTileKeys;
            const long long cost = whole ? 1 : k.nt + kUnitCost, from = u0, u1 = min(cost, u0 + (x1 - x));
            unit_at = x - u0;
            x += u1 - u0;
            if (u1 == cost) { ++qt; u0 = 0; } else u0 = u1;
            if (piece_tiles(from, whole ? k.nt : u1, cta, k)) return true;
        }
        return false;
    }
};

// The last request with cu[r] <= t, by one warp: two rounds of loads for up to 1024 requests.
__device__ __forceinline__ int find_request(const PagedAttnArgs& p, int t, int lane) {
    const int step = (p.R + 31) / 32, i = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < p.R && p.cu[i] <= t);
    int r = (31 - __clz(m | 1u)) * step;
    if (step == 1) return r;
    const int end = min(r + step, p.R);
    for (int base = r; base < end; base += 32) {
        const unsigned b = __ballot_sync(0xffffffffu, base + lane < end && p.cu[base + lane] <= t);
        if (b) r = base + 31 - __clz(b);
        if (b != 0xffffffffu) break;
    }
    return r;
}

// Selected blocks: whole units (KV head, token) round the CTAs, then the piece [x, x1) of
// the line of the units left over.  Run by one warp, which compacts a unit's valid blocks
// into the list.
struct WalkSel {
    long long unit, rounds_end, x, x1, total, pieces, unit_at;
    __device__ __forceinline__ void start(const Params& P, int cta, int grid) {
        const long long units = (long long)P.a.T * P.a.hkv;
        unit = cta;
        rounds_end = P.whole_sel ? units : units - units % grid;
        total = (units - rounds_end) * P.cost_sel;
        pieces = min((long long)grid, total);
        x = cta < pieces ? quotient(cta * total, pieces) : 0;
        x1 = cta < pieces ? quotient((cta + 1) * total, pieces) : 0;
    }
    __device__ __forceinline__ bool next(const Params& P, int cta, int grid, int lane, int* list, Piece& k) {
        const PagedAttnArgs& p = P.a;
        const int t_first = p.cu[0], t_last = p.cu[p.R];
        for (;;) {
            long long u, u0 = 0, u1 = P.cost_sel;
            if (unit < rounds_end) {
                u = unit;
                unit += grid;
            } else if (x < x1) {
                const long long i = quotient(x, P.cost_sel);
                u0 = x - i * P.cost_sel;
                u1 = min(u1, u0 + (x1 - x));
                u = rounds_end + i;
                unit_at = x - u0;
                x += u1 - u0;
            } else {
                return false;
            }
            const int g = (int)quotient(u, p.T), t = (int)(u - (long long)g * p.T);
            if (t < t_first || t >= t_last) continue;
            const int32_t* row = p.bidx + ((long long)t * p.hkv + g) * p.topk;
            const int b0 = lane < p.topk ? row[lane] : -1;
            const int b1 = lane + 32 < p.topk ? row[lane + 32] : -1;
            k.r = find_request(p, t, lane);
            const Req q = request(p, k.r);
            if (t < q.a || t >= q.a + q.n) continue;
            int nt;
            unit_keys(q, t - q.a, 1, p.swin, &k.pos0, &k.lo, &k.hi, &nt);
            const int pos = k.pos0, qb = pos >= 0 ? pos / p.bs : -1;
            const unsigned m0 = __ballot_sync(0xffffffffu, block_valid(b0, qb, pos, p.bs, p.swin));
            const unsigned m1 = __ballot_sync(0xffffffffu, block_valid(b1, qb, pos, p.bs, p.swin));
            const unsigned below = (1u << lane) - 1u;
            if (m0 >> lane & 1) list[__popc(m0 & below)] = b0;
            if (m1 >> lane & 1) list[__popc(m0) + __popc(m1 & below)] = b1;
            __syncwarp();
            k.nb = __popc(m0) + __popc(m1);
            k.tok0 = t;
            k.ntok = 1;
            k.g = g;
            const int per = kTileKeys / p.bs;
            k.nt = (k.nb + per - 1) / per;
            if (piece_tiles(u0, u1, cta, k)) return true;
        }
    }
};

// The visible columns of key tile j of a piece, as two inclusive ranges: columns
// [l0, h0] of the first 64 and [l1, h1] of the last 64 (empty: l > h).  For the unit as a
// whole; rows narrow them further.
template <bool SEL>
__device__ __forceinline__ void tile_cols(const Params& P, const Piece& k, const int* list, int j, int& l0,
                                          int& h0, int& l1, int& h1) {
    if (!SEL) {
        const int key0 = (k.tile0 + j) * kTileKeys;
        l0 = max(k.lo - key0, 0);
        h1 = min(k.hi - key0, 127);
        h0 = min(h1, 63);
        l1 = max(l0, 64);
    } else if (P.a.bs == 128) {
        const int key0 = list[j] * 128;
        l0 = max(k.lo - key0, 0);
        h1 = min(k.hi - key0, 127);
        h0 = min(h1, 63);
        l1 = max(l0, 64);
    } else {
        const int key0 = list[2 * j] * 64;
        l0 = max(k.lo - key0, 0);
        h0 = min(k.hi - key0, 63);
        l1 = 128;
        h1 = -1;
        if (2 * j + 1 < k.nb) {
            const int key1 = list[2 * j + 1] * 64;
            l1 = 64 + max(k.lo - key1, 0);
            h1 = 64 + min(k.hi - key1, 63);
        }
    }
}

// The stages of the K and V tiles: kRings rings of kPer stages.  One ring where both issuers
// use every tile; one per stream, tile t in ring t & 1, where the streams take turns: a stage
// then has one issuer to wait for it, and no wait can be a phase behind (with one ring and a
// stage count that is no multiple of 4, the streams would take turns on a stage, and the one
// ahead could take the phase before its own for its own).  A ring's places go in the order
// of use: kAhead K tiles, then V and K in turn.
template <int kRings, int kPer, int kAhead>
struct Ring {
    static constexpr int kRun = kRings * kAhead;     // K tiles loaded ahead of V, over all rings
    struct At { int stage; uint32_t phase; };
    __device__ __forceinline__ static uint32_t phase(int place) { return (uint32_t)(place / kPer) & 1u; }
    __device__ __forceinline__ static At at(int t, int place) {
        return {(kRings == 2 ? (t & 1) * kPer : 0) + place % kPer, phase(place)};
    }
    __device__ __forceinline__ static int k_place(int t) {
        const int i = kRings == 2 ? t >> 1 : t;
        return i < kAhead ? i : 2 * i - kAhead + 1;
    }
    __device__ __forceinline__ static int v_place(int t) { return 2 * (kRings == 2 ? t >> 1 : t) + kAhead; }
    __device__ __forceinline__ static At k(int t) { return at(t, k_place(t)); }
    __device__ __forceinline__ static At v(int t) { return at(t, v_place(t)); }
};

// Bounded wait of a whole warp; false in every lane if any lane gave up.  A role that finds
// nothing to wait for goes on whether or not another has given up; one that has to wait then gives
// up too.  (Looking at the flag before every wait, and in the loop: selected blocks of a chunk of
// 512 tokens 304 us, in the loop alone 288; 64 bits of the clock: 291.)
static_assert(kWaitBudgetCycles < (1ll << 32), "the waits count cycles in 32 bits");
struct Waiter {
    volatile int* abort_flag;
    int* err;
    __device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        const uint32_t start = (uint32_t)clock();
#pragma unroll 1
        while (!mbar_try_wait(bar, parity)) {
            if (*abort_flag) return false;
            if ((uint32_t)clock() - start > (uint32_t)kWaitBudgetCycles) {
                *err = NSA_ERR_TIMEOUT;
                *abort_flag = 1;
                return false;
            }
        }
        return true;
    }
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, lane_wait(bar, parity));
    }
};

// One status byte per CTA, always written: nothing has to be cleared before the call.
__device__ __forceinline__ void finish_status(DevStatus* st, int err, int cta, int grid) {
    cta_status(st)[cta] = (unsigned char)err;
    if (cta == 0) {
        st->code = 0;
        st->index_tag = 0;      // an index inversion left in this workspace is gone
        for (int i = grid; i < kMaxStatusCtas; ++i) cta_status(st)[i] = 0;
    }
}

// Piece i of the scheduler's ring, once it is there; release: this warp is done with it.
template <class Smem>
__device__ __forceinline__ bool fetch_piece(Smem& S, const Waiter& wait, int i) {
    return wait(&S.ring_full[i % kRing], (i / kRing) & 1);
}
template <class Smem>
__device__ __forceinline__ void release_piece(Smem& S, int lane, int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.ring_empty[i % kRing]);
}

// A unit that sees no key: out = 0, lse = -inf, by one warp.
__device__ __forceinline__ void write_empty(const PagedAttnArgs& p, const Piece& k, int lane) {
    for (int t = k.tok0; t < k.tok0 + k.ntok; ++t) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)t * p.hq + k.g * p.G) * p.d);
        for (int i = lane; i < p.G * p.d / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = lane; h < p.G; h += 32) p.lse[(size_t)(k.g * p.G + h) * p.T + t] = -CUDART_INF_F;
    }
}

// The scheduler warp: walks the CTA's pieces of work ahead of the others.  Every piece in the
// ring has a key tile: units that see no key are written here.  (An issuer looks ahead for its
// next S but gives a place of the ring back with its P V, so that a run of pieces without a
// tile could fill the ring before it finds one, and nobody could go on.)
template <bool SEL, class Smem>
__device__ __forceinline__ void schedule(Smem& S, const Params& P, const Waiter& wait, int tpu, int cta, int grid,
                                         int lane) {
    const PagedAttnArgs& p = P.a;
    WalkAll wall{};
    WalkSel wsel{};
    if (SEL) {
        wsel.start(P, cta, grid);
        bool good = true;
        if (cta == 0)
            for (int r = lane; r < p.R; r += 32) good &= request_ok(p, r);
        if (!good) S.err = NSA_ERR_BAD_INDEX;
    } else if (!wall.start(P, tpu, cta, grid, lane)) {
        S.err = NSA_ERR_BAD_INDEX;
    }
    // the unit this CTA starts and leaves open, for the merge, and who finishes it
    int4 open = make_int4(0, 0, 0, -1);
    for (int i = 0;; ++i) {
        const int at = i % kRing;
        if (!wait(&S.ring_empty[at], ((i / kRing) & 1) ^ 1)) break;
        Piece k{};
        for (bool more = true; more;) {
            more = SEL ? wsel.next(P, cta, grid, lane, S.list[at], k) : wall.next(P, tpu, cta, k);
            if (!more) k.more = 0;
            else if (k.nt == 0) write_empty(p, k, lane);
            else break;
        }
        if (k.more && k.slot == 2 * cta + 1)     // its last key tile's place on the line
            open = make_int4(k.tok0, k.ntok, k.g,
                             SEL ? owner_of(wsel.unit_at + k.nt - 1, wsel.total, wsel.pieces)
                                 : owner_of(wall.unit_at + k.nt - 1, wall.total, wall.pieces));
        if (lane == 0) S.ring[at] = k;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.ring_full[at]);
        if (!k.more) break;
    }
    if (lane == 0) P.desc[cta] = open;
}

// The producer warp: each unit's Q (kTiles tiles of query rows), and its K and V tiles page by
// page through the block table, one lane per box.
template <bool SEL, int kTiles, class Stages, class Smem>
__device__ __forceinline__ void produce(Smem& S, const Params& P, const Waiter& wait, const CUtensorMap* qmap,
                                        const CUtensorMap* kmap, const CUtensorMap* vmap, int lane) {
    constexpr int kHalves = Smem::kHalves, kRun = Stages::kRun;
    const PagedAttnArgs& p = P.a;
    const int boxes = kTileKeys / P.box_rows;      // per tile: at most 16
    const uint32_t box_bytes = (uint32_t)P.box_rows * (kHalves * 128u);
    // (page and block sizes are powers of two)
    const int ps_log2 = 31 - __clz(p.ps), bs_log2 = SEL ? 31 - __clz(p.bs) : 0;
    const int c0 = lane * P.box_rows;              // this lane's box: its first key in the tile
    int tk = 0, tv = 0;         // K and V tiles loaded
    int units = 0;              // units whose Q was loaded
    int at = -1;                // piece of the next K tile
    int j = 0, j_end = 0;       // the key tile after it
    bool ok = true, more = true, new_unit = false;
    // The next K tile's box of this lane.  It is looked up one tile ahead: the block table's
    // entry comes from L2 or memory, and would hold up every tile.
    bool nx_live = false;
    int nx_page = 0, nx_row = 0, nx_g = 0;
    auto advance = [&]() -> bool {
        if (j == j_end) {                     // the next piece
            if (at >= 0) release_piece(S, lane, at);
            if (!fetch_piece(S, wait, ++at)) return false;
            const Piece& k = S.ring[at % kRing];
            more = k.more != 0;
            j = k.p0;
            j_end = k.p1;
            new_unit = true;
        }
        if (!more) return true;
        const Piece& k = S.ring[at % kRing];
        int key = -1;
        if (lane < boxes) {
            if (!SEL) {
                key = (k.tile0 + j) * kTileKeys + c0;
            } else {
                const int e = ((j * kTileKeys) >> bs_log2) + (c0 >> bs_log2);
                if (e < k.nb) key = (S.list[at % kRing][e] << bs_log2) + (c0 & (p.bs - 1));
            }
        }
        nx_live = key >= 0 && key <= k.hi && key + P.box_rows > k.lo;   // a visible key lies in it
        nx_row = key & (p.ps - 1);
        nx_g = k.g;
        if (nx_live) nx_page = p.table[(long long)k.r * p.table_stride + (key >> ps_log2)];
        ++j;
        return true;
    };
    // the tiles whose K is on its way and whose V is not: the boxes' coordinates
    int key_q[kRun] = {}, group_q[kRun] = {}, last_q[kRun] = {};
    unsigned mask_q[kRun] = {};
    int pending = 0;
    auto load = [&](const CUtensorMap* map, typename Stages::At to, int c1, int c3, int c4, unsigned mask) -> bool {
        const int stg = to.stage;
        if (!wait(&S.kv_empty[stg], to.phase ^ 1)) return false;
        if (lane == 0) mbar_arrive_expect_tx(&S.kv_full[stg], (uint32_t)__popc(mask) * box_bytes);
        __syncwarp();
        if (mask >> lane & 1)
            tma_load_rows(S.kv[stg] + lane * box_bytes, map, &S.kv_full[stg], c1, c3, c4);
        return true;
    };
    ok = advance();
    while (ok) {
        if (more) {
            if (new_unit) {
                const Piece& k = S.ring[at % kRing];
                const int qb = kTiles == 2 ? 0 : units & 1;
                const int use = kTiles == 2 ? units : units >> 1;
                if (!(ok = wait(&S.q_empty[qb], (use & 1) ^ 1))) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(&S.q_full[qb], (uint32_t)(kTiles * kHalves * P.tpt * p.G) * 128u);
                __syncwarp();
                if (lane < kTiles * kHalves) {
                    const int tile = lane / kHalves, hf = lane - tile * kHalves;
                    tma_load_3d(S.q[kTiles == 2 ? tile : qb][hf], qmap, &S.q_full[qb], hf * 64, k.g * p.G,
                                k.tok0 + tile * P.tpt);
                }
                ++units;
                new_unit = false;
            }
            if (nx_live && (nx_page < 0 || nx_page >= p.num_pages)) {   // reads as zeros
                S.err = NSA_ERR_BAD_INDEX;
                nx_page = p.num_pages;
            }
            const unsigned mask = __ballot_sync(0xffffffffu, nx_live);
            const int c1 = P.page_groups ? 0 : nx_row;
            const int c3 = P.page_groups ? nx_page * P.page_groups + (nx_row >> 3) : nx_g;
            const int c4 = P.page_groups ? nx_g : nx_page;
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (i == pending) {
                    key_q[i] = c1;
                    group_q[i] = c3;
                    last_q[i] = c4;
                    mask_q[i] = mask;
                }
            if (!(ok = load(kmap, Stages::k(tk), c1, c3, c4, mask))) break;
            ++tk;
            ++pending;
            if (!(ok = advance())) break;
            if (pending < kRun) continue;
        }
        if (pending == 0) break;
        if (!(ok = load(vmap, Stages::v(tv), key_q[0], group_q[0], last_q[0], mask_q[0]))) break;
        ++tv;
#pragma unroll
        for (int i = 0; i + 1 < kRun; ++i) {
            key_q[i] = key_q[i + 1];
            group_q[i] = group_q[i + 1];
            last_q[i] = last_q[i + 1];
            mask_q[i] = mask_q[i + 1];
        }
        --pending;
    }
    if (lane == 0) {
        S.loaded[0] = tk;
        S.loaded[1] = tv;
        S.loaded[2] = units;
    }
    __syncwarp();
}

// Where a role gave up, copies may be in flight that nobody waits for: they land before the CTA
// exits.  By the producer warp, when every role has ended; a lane per stage, for its last copy.
template <int kTiles, class Stages, class Smem>
__device__ __forceinline__ void land_copies(Smem& S, int lane) {
    const int tk = S.loaded[0], tv = S.loaded[1], units = S.loaded[2];
    int place = -1;
    for (int t = max(tk - 2 * Smem::kStages, 0); t < tk; ++t) {
        const int k = Stages::k_place(t), v = t < tv ? Stages::v_place(t) : -1;
        if (Stages::at(t, k).stage == lane) place = max(place, k);
        if (v >= 0 && Stages::at(t, v).stage == lane) place = max(place, v);
    }
    uint64_t* bar = nullptr;
    uint32_t parity = 0;
    if (lane < Smem::kStages) {
        if (place >= 0) bar = &S.kv_full[lane];
        parity = Stages::phase(place);
    } else if (lane < Smem::kStages + 2) {
        const int i = lane - Smem::kStages;
        const int uses = kTiles == 2 ? (i == 0 ? units : 0) : (units + 1 - i) / 2;
        if (uses > 0) bar = &S.q_full[i];
        parity = (uint32_t)(uses - 1) & 1u;
    }
    const uint32_t start = (uint32_t)clock();
    while (bar && !mbar_try_wait(bar, parity) && (uint32_t)clock() - start < (uint32_t)(kWaitBudgetCycles / 64)) {}
    __syncwarp();
}

// paged_few.cu: units of at most kFewRows query rows.
constexpr int kFewRows = 16;
cudaError_t launch_paged_few(const Params& P, int f16, int grid, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, cudaStream_t stream);

}  // namespace nsa
