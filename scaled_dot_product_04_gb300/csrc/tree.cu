// Attention of each request's new tokens (one token, a drafted tree, or a
// chunk of a prompt) over its paged key/value cache:
//
//   O_i = sum_j p_ij V_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - m_i),
//   LSE_i = m_i + ln sum_j p_ij,
//
// over the keys j that row i sees: every key of the context, and those of the
// request's own new tokens that its mask row names (with no mask: itself and
// the ones before it).
//
// What bounds it.  A request's keys and values are read once for the rows of
// one key/value head, n tokens x (h / h_kv) query heads: 4 d rows operations
// for 4 d bytes of a 16-bit key and value, so below some 280 rows the memory
// is the floor, and the whole design serves the loads.
//
// Rows are the M side of both products, S = Q K^T and O += P V, as in the
// dense forward (fwd_pair.cu), whose two chains x = 0, 1 of S_x, P_x, O_x in
// TMEM, one MMA-issuing thread and two softmax warpgroups this kernel shares.
// A unit is a row tile of one request and key/value head; kRows is the most
// rows a tile holds, chosen by the host from the longest request:
//   256     a unit of more than 128 rows has rows 128 x .. 128 x + 127 in chain
//           x and both chains read every key tile (`both`); in one of fewer
//           rows the chains take its key tiles in turn, so two softmaxes work
//           at a time;
//   64, 32  in turn as well, and the TMEM lanes are split: the rows are repeated
//           2 or 4 times down the 128 lanes, and each repeat exponentiates its
//           own half or quarter of the tile's keys and leaves zeros at the
//           others' (P V sums over all keys; the product's time does not depend
//           on the rows, and the loads cover it).  A warp then has 64 or 32 keys
//           a row to exponentiate instead of 128.
// Each chain and repeat keeps a running maximum and sum of its own; they are
// joined when the unit ends.
//
// Schedule.  The units' key tiles, request by request, form one list whose
// length every CTA computes from the lengths on the device, and CTA c of G runs
// the c-th of G equal shares: ragged lengths balance to a tile or two, and a few
// long requests fill the GPU.  A unit that a CTA does not run from its first to
// its last tile leaves its sums, maximum and unscaled O in the workspace (two
// parts a CTA at most), and a second small kernel joins the parts in their
// order, so results do not change from run to run.
//
// Measured (GB300; b requests x n tokens, 32 heads on 8, d = 128; of the copy
// rate 6.78 TB/s): 64 x 1, 200-8100 keys, bf16: 168 us, 98%.  16 x 32, 500-16000
// keys: 99 us, 85%, of which the joining takes 6.  8 x 64 over 8000-32000 keys,
// fp16: 134 us, 67% and 1.14 PFLOP/s, joining 6; 4 x 500 after 2000-12000: 76 us,
// 0.91 PFLOP/s, joining 9: the tensor pipe is busy 57% and 47% of the main kernel's
// time, the DRAM 64% and 28%, so neither is the limit; which of S, softmax and P V
// a chain waits for has not been taken apart.  32 x 13, E4M3: 105 us, 73%: tensor
// pipe 56%, DRAM 66%.
// Tried and slower: tiles asked into L2 two, four or eight ahead of the ring
// (64 x 1: 175 -> 190, 230, 279 us); the joining by whichever CTA is last,
// inside this kernel (its code is cold when it runs, +6 us and more); short
// units kept whole to spare the joining (1 request of 1000 keys 11.3 -> 14.2).
//
// Roles: warp 0 loads K and V tiles (a lane a page and 128-byte column), warp
// 1 issues the products, warps 2 and 3 load Q, warps 4-7 and 8-11 are the two
// chains' softmax.
//
// 16-bit caches.  P enters P V in the cache's type, which is what the product
// takes beside V: off by 2^-8 (bf16) or 2^-11 (fp16) of itself, while its sum is
// kept in fp32.  Against 64 bits O is off by 0.0022 and 0.00029, where rounding O
// alone leaves 0.0017 and 0.00021.
//
// E4M3 caches.  The tiles stay in 8 bits; Q and P enter as sums of 8-bit terms
// instead.  Q's row is scaled by a power of two to at most 2^8 and written as
// E4M3 hi + lo (+ lo2 for fp16, whose 11 bits need three): exact down to 2^-17
// of the row's largest value.  P, raised by 2^8, is written as E5M2 hi, rounded,
// and the rest as E4M3 lo: hi leaves at most 2^-3 of the power of two below P,
// of which lo leaves 2^-4, so P is off by 2^-7 of itself; for fp16 another
// 2^-4 of that goes to an E4M3 lo2, which leaves 2^-11, fp16's own half step
// (O off by 0.00028 and not 0.0012).  lo's smallest step ends that at 2^-11
// (2^-7 for fp16) of the row's largest weight: from there on weights are off by
// up to 2^-18 of the largest, though never more than hi's 2^-3 of themselves.
// (With an E4M3 hi, those below 2^-17 would vanish, and a long context has very
// many of them.)  The terms cost products and conversions, so the 8-bit cache
// pays where the memory is the limit and not for many rows (us, bf16 /
// fp16 over E4M3 beside the 16-bit cache): 64 x 1 102 / 127 beside 171, 16 x 32 89
// beside 99; but 4 x 500 108 / 137 beside 74, 8 x 64 215 (fp16) beside 123.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache.cuh"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;  // 65536 / 384, rounded down to a multiple of 8
constexpr uint32_t kRegsWg0 = 104, kRegsSoftmax = 200;
static_assert(kRegsWg0 + 2 * kRegsSoftmax == 3 * kLaunchRegs, "the split must hand out the launch's registers");
constexpr float kLn2 = 0.693147180559945309f;

template <int D, bool kFp8, int kRows>
struct TreeLayout {
    static constexpr bool kPair = kRows == 256;               // a unit's rows may need both chains
    static constexpr int kSplit = kPair ? 1 : 128 / kRows;    // repeats of the rows down the lanes
    static constexpr int kUnique = 128 / kSplit;              // rows of one chain and repeat
    static constexpr int kEb = kFp8 ? 1 : 2;
    static constexpr int kChunks = D * kEb / 128;
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kQTerms = kFp8 ? 3 : 1;               // Q tiles of a chain
    static constexpr int kQBytes = kQTerms * kTileBytes;
    static constexpr int kQTiles = kPair ? 2 : 1;
    static constexpr int kStages = kTileBytes == 32768 ? 5 : kFp8 && kPair ? 7 : 8;
    static constexpr int kUnitCost = kPair ? (kFp8 ? 5 : 4) : kFp8 ? 4 : kSplit == 4 ? 1 : 3;  // see unit_places
    static constexpr int kQ = 0;
    static constexpr int kRing = kQ + kQTiles * kQBytes;
    // joining the repeats: a warp's columns for the other repeats' warps
    static constexpr int kOwn = D / 2 / kSplit;               // columns that a warp writes out
    static constexpr int kGive = kSplit == 4 ? kOwn / 2 : kOwn;  // of which it takes or gives so many at a time
    static constexpr int kJoin = kRing + kStages * kTileBytes;
    static constexpr int kStats = kJoin + 8 * 32 * (kSplit - 1) * kGive * 4;  // float2 (base, l) [2][128]
    static constexpr int kQScale = kStats + 2 * 128 * 8;      // float [256]: 1 / Q's row scale
    static constexpr int kScan = kQScale + (kFp8 ? 256 * 4 : 0);  // int64 [12], the start record
    static constexpr int kBar = kScan + 12 * 8 + 48;
    static constexpr int bFull = 0;
    static constexpr int bEmpty = bFull + kStages;
    static constexpr int bQFull = bEmpty + kStages;
    static constexpr int bQEmpty = bQFull + 1;
    static constexpr int bSFull = bQEmpty + 1;   // + x
    static constexpr int bPReady = bSFull + 2;
    static constexpr int bOFull = bPReady + 2;
    static constexpr int bOFree = bOFull + 2;
    static constexpr int bJoin = bOFree + 2;
    static constexpr int bMmaIdle = bJoin + 1;
    static constexpr int kNumBars = bMmaIdle + 1;
    static constexpr int kMisc = kBar + kNumBars * 8;  // u32[0] TMEM base, u32[1] abort flag
    static constexpr int kBytes = kMisc + 16;
    static_assert(kBytes <= 232448, "tree kernel exceeds shared memory");
    static constexpr uint32_t kColS = 0, kColO = 256;  // S_x at 128 x, O_x at 256 + D x
    // workspace: parts of kRows rows, O then (base, l); two a CTA
    static constexpr size_t kPartFloats = (size_t)kRows * (D + 2);
};

SDPA_DEV bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx &w, uint32_t site) {
    bool ok = mbar_wait(bar, parity, w, site);
    return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ schedule
// Tokens of a row tile; of one chain's share of it: chain_tokens.
template <int kRows>
__host__ __device__ inline int tokens_per_tile(const TreeParams &p) {
    return (kRows == 256 ? 2 : 1) * p.chain_tokens;
}

// One request as every role sees it; lengths are clamped so that whatever the
// arrays hold, reads and writes stay inside q, o, the table and the cache.
struct Request {
    int q0, n, ctx, end, tiles;  // first token, tokens, context keys, keys to read, row tiles
};
template <int kRows>
SDPA_DEV Request load_request(const TreeParams &p, int b) {
    Request r;
    r.q0 = min(max(p.cu_q[b], 0), p.total_q);
    r.n = max(min(p.cu_q[b + 1], p.total_q) - r.q0, 0);
    const int len = max(p.kv_lens[b], 0);
    r.ctx = len - r.n;
    r.end = min(min(len, p.max_kv), p.max_blocks * p.page_size);
    const int per = tokens_per_tile<kRows>(p);
    r.tiles = r.n <= per ? min(r.n, 1) : (r.n + per - 1) / per;
    return r;
}
// Keys that row tile rt reads (a chain's rows see nothing behind the last of them), and its key tiles.
template <int kRows>
SDPA_DEV int tile_end(const TreeParams &p, const Request &r, int rt) {
    if (p.mask) return r.end;
    return max(min(r.end, r.ctx + min(r.n, (rt + 1) * tokens_per_tile<kRows>(p))), 0);
}
SDPA_DEV int key_tiles(int end) { return max((end + kTileN - 1) / kTileN, 1); }
// The shared list.  A unit has a place for each key tile, or two where both
// chains read every tile (such a tile takes almost twice as long unless the
// memory is the limit), and before them `cost` places: about what starting and
// ending a unit takes in a CTA.  A CTA runs the tiles that end in its share, so
// a unit's first CTA is the one whose share holds the end of its first tile.
template <int kRows>
SDPA_DEV int tile_places(const TreeParams &p, const Request &r, int rt) {
    return kRows == 256 && r.n - rt * tokens_per_tile<kRows>(p) > p.chain_tokens ? 2 : 1;
}
template <int kRows>
SDPA_DEV int unit_places(const TreeParams &p, const Request &r, int rt, int cost) {
    return cost + tile_places<kRows>(p, r, rt) * key_tiles(tile_end<kRows>(p, r, rt));
}
template <int kRows>
SDPA_DEV int64_t head_places(const TreeParams &p, const Request &r, int cost) {
    // with a mask every row tile reads all keys, and all but the last are alike
    if (p.mask && r.tiles > 0)
        return (int64_t)(r.tiles - 1) * unit_places<kRows>(p, r, 0, cost) + unit_places<kRows>(p, r, r.tiles - 1, cost);
    int64_t sum = 0;
    for (int rt = 0; rt < r.tiles; ++rt) sum += unit_places<kRows>(p, r, rt, cost);
    return sum;
}

// A CTA's walk over its share: unit after unit, each with a first and last tile.
struct Start {
    int left;            // places of this CTA (the host bounds the list to 31 bits)
    int b, head, rt, t;  // where its first place lies
    Request r;           // request b
};
struct Piece {
    int b, head;         // request, key/value head
    int q0, ctx, end;    // of the request; end of the row tile
    int tok, ntok;       // the row tile's first token (in the request) and tokens
    int unit_tiles, ta, tb;
};
template <int kRows, int cost>
struct Walk {
    const TreeParams &p;
    Request r;
    int b, head, rt, t, left;
    SDPA_DEV Walk(const TreeParams &p_, const Start &s)
        : p(p_), r(s.r), b(s.b), head(s.head), rt(s.rt), t(s.t), left(s.left) {}
    SDPA_DEV bool next(Piece &u) {
        while (left > 0) {
            while (rt >= r.tiles) {  // the head's or request's last row tile is done
                rt = 0;
                if (++head < p.h_kv && r.tiles > 0) continue;
                head = 0;
                if (++b >= p.num_seqs) return false;
                r = load_request<kRows>(p, b);
            }
            const int per = tokens_per_tile<kRows>(p), wide = tile_places<kRows>(p, r, rt);
            u.b = b;
            u.head = head;
            u.q0 = r.q0;
            u.ctx = r.ctx;
            u.end = tile_end<kRows>(p, r, rt);
            u.tok = rt * per;
            u.ntok = min(per, r.n - u.tok);
            u.unit_tiles = key_tiles(u.end);
            const int places = min(cost + wide * u.unit_tiles, t + left);
            // tiles that end before t, and before the share's end (a shift: wide is 1 or 2)
            u.ta = max(t - cost, 0) >> (wide - 1);
            u.tb = max(places - cost, 0) >> (wide - 1);
            left -= places - t;
            t = 0;
            ++rt;
            if (u.tb > u.ta) return true;  // a share may begin or end beside a tile's end
        }
        return false;
    }
};

// Order of a piece's n key tiles in the ring, by how far S runs ahead of P V: K_0 V_0 K_1 V_1 ..
// where both chains read every tile, K_0 K_1 V_0 K_2 V_1 .. V_{n-1} where they take turns.  V_i
// and the K behind it land on one barrier (V_i's), so the issuing thread waits once for both.
SDPA_DEV int k_pos(bool both, int i) { return both ? 2 * i : i == 0 ? 0 : 2 * i - 1; }
SDPA_DEV int v_pos(bool both, int i, int n) { return both ? 2 * i + 1 : i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// Bits of the 32 keys from `key` that token i of the request sees (a key
// behind `end` is not there).
SDPA_DEV uint32_t seen_bits(const TreeParams &p, const Piece &u, int i, int key) {
    const int have = u.end - key;  // keys that are there
    const uint32_t there = have >= 32 ? 0xffffffffu : have <= 0 ? 0u : (1u << have) - 1u;
    const int t = key - u.ctx;     // number of the first key among the new tokens
    if (!p.mask) {
        const int upto = i + 1 - t;
        return there & (upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u);
    }
    if (t <= -32) return there;
    const uint32_t *row = p.mask + (int64_t)(u.q0 + i) * p.mask_words;
    const int w = t >> 5;  // may be -1: the context's keys, all seen
    const uint32_t lo = w < 0 ? 0xffffffffu : w < p.mask_words ? row[w] : 0u;
    const uint32_t hi = w + 1 < p.mask_words ? row[w + 1] : 0u;
    return there & __funnelshift_r(lo, hi, t & 31);
}

// Workspace record of a unit that CTA c finds already begun: how its parts join.
struct Cut {
    int16_t parts;  // 0: CTA c finds none begun
    int16_t mine;   // CTA c is the mine-th (from 0) to continue it
    int q_tok, ntok, head;
};

// ------------------------------------------------------------------ kernel
template <int D, int kEl, bool kFp8, int kRows>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using L = TreeLayout<D, kFp8, kRows>;
    constexpr bool kBf16 = kEl == kElBf16;
    constexpr int kSplit = L::kSplit;
    constexpr bool kPair = L::kPair;
    constexpr int kQTerms = kFp8 ? (kBf16 ? 2 : 3) : 1, kPTerms = kQTerms;
    constexpr int cost = L::kUnitCost;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {  // the tiles' swizzle counts on it
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, (kTagTree << 16) | 20u);
        return;
    }
    auto bar = [&](int i) -> uint32_t { return sbase + L::kBar + 8u * i; };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    const uint32_t warp = warp_id(), lane = lane_id();
    Cut *cuts = reinterpret_cast<Cut *>(p.workspace);
    float *parts = reinterpret_cast<float *>(p.workspace + kTreeMaxCtas * sizeof(Cut));

    Start *start = reinterpret_cast<Start *>(smem + L::kScan + 12 * 8);
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar(L::bFull + s), 1);
            mbar_init(bar(L::bEmpty + s), 1);
        }
        mbar_init(bar(L::bQFull), kFp8 ? 2 : 1);      // the two Q warps, or the load
        mbar_init(bar(L::bQEmpty), kFp8 ? 9 : 1);     // the last S; the 8 softmax warps have the row scales
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(L::bSFull + x), 1);
            mbar_init(bar(L::bPReady + x), 4);
            mbar_init(bar(L::bOFull + x), 1);
            mbar_init(bar(L::bOFree + x), 8);
        }
        mbar_init(bar(L::bJoin), 8);
        mbar_init(bar(L::bMmaIdle), 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(sbase + L::kMisc, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        if (!kFp8) tma_prefetch_desc(&tm_q);
    }
    griddep_wait();  // nothing of the caller's is read or written before this

    // ---- this CTA's share of the tile list
    int64_t *scan = reinterpret_cast<int64_t *>(smem + L::kScan);

    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min(p.num_seqs, (int)threadIdx.x * per), b1 = min(p.num_seqs, b0 + per);
    int64_t sum = 0, one = 0;  // one: of the thread's first request, mostly its only one
    Request r{};
    for (int b = b0; b < b1; ++b) {
        const Request q = load_request<kRows>(p, b);
        const int64_t places = head_places<kRows>(p, q, cost);
        if (b == b0) {
            r = q;
            one = places;
        }
        sum += p.h_kv * places;
    }
    int64_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if ((int)lane >= off) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (int)warp) before += scan[w];
        total += scan[w];
    }
    // a share is no less than a tile, so every CTA between a unit's first and last runs one of its tiles
    const int ctas = total > 0 ? (int)min((int64_t)gridDim.x, max(total / (kPair ? 2 : 1), (int64_t)1)) : 0, c = blockIdx.x;
    if (c < ctas) {
        // CTA i has places [begin(i), begin(i + 1))
        const int64_t each = total < INT32_MAX ? (int)total / ctas : total / ctas;
        const int more = (int)(total - each * ctas);
        auto begin = [&](int i) { return each * i + min(i, more); };
        const int64_t first = begin(c);
        if (first >= before && first < before + sum) {  // this thread's requests hold the first place
            int b = b0;
            int64_t at = first - before;
            int64_t ht = one;
            while (at >= p.h_kv * ht) {
                at -= p.h_kv * ht;
                r = load_request<kRows>(p, ++b);
                ht = head_places<kRows>(p, r, cost);
            }
            int head = 0, rt = 0, places = unit_places<kRows>(p, r, 0, cost);
            while (at >= ht) {
                at -= ht;
                ++head;
            }
            while (at >= places) {
                at -= places;
                places = unit_places<kRows>(p, r, ++rt, cost);
            }
            *start = Start{(int)(begin(c + 1) - first), b, head, rt, (int)at, r};
            Cut cut{0, 0, 0, 0, 0};
            const int64_t unit0 = first - at, unit1 = unit0 + places;
            const int64_t tile1 = unit0 + cost + tile_places<kRows>(p, r, rt);  // behind the first tile
            if (first >= tile1) {  // a CTA before this one has the unit's first tile
                const int tpt = tokens_per_tile<kRows>(p);
                int i = c, j = c + 1;  // the first to continue it; the first behind it
                while (begin(i - 1) >= tile1) --i;
                while (j < ctas && begin(j) < unit1) ++j;
                cut.parts = (int16_t)(j - i + 1);
                cut.mine = (int16_t)(c - i);
                cut.q_tok = r.q0 + rt * tpt;
                cut.ntok = min(tpt, r.n - rt * tpt);
                cut.head = head;
            }
            cuts[c] = cut;
        }
    } else if (threadIdx.x == 0) {  // fewer places than CTAs
        cuts[c].parts = 0;
        *start = Start{};
    }
    // Each role waits for the start record in its own code (the same barrier, met by every warp
    // once), so its first instructions are fetched while the record is made.
    const WaitCtx wc{reinterpret_cast<volatile uint32_t *>(&misc[1]), p.err, kTagTree};
    using Units = Walk<kRows, cost>;
    Piece u;

    if (warp < 4) {
        setmaxnreg_dec<kRegsWg0>();
        if (warp == 0) {
            // ======================================================== K and V
            // a tile is `pages` boxes of `box` rows; lane = page * kChunks + 128-byte column
            const int box = min(p.page_size, kTileN), pages = p.page_size < kTileN ? kTileN >> p.page_shift : 1;
            const int mine = (int)lane / L::kChunks, col = (int)lane % L::kChunks;
            const bool loads = mine < pages;
            const int none = p.num_pages * p.h_kv;  // behind the last: reads as zeros
            const int tpc = p.chain_tokens;
            uint32_t stage = 0, phase = 0;  // the ring's next place
            bool ok = true;
            __syncthreads();
            Units walk(p, *start);
            while (ok && walk.next(u)) {
                const int n = u.tb - u.ta;
                // (y, z) of this lane's box of the piece's tile i
                auto place = [&](int i, int &y, int &z) {
                    y = 0;
                    z = none;
                    if (!loads || i >= n) return;
                    const int key = (u.ta + i) * kTileN + mine * box;
                    if (key >= u.end) return;
                    const int blk = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
                    const int page = p.table[(int64_t)u.b * p.max_blocks + blk];
                    y = key - blk * p.page_size;
                    if (page >= 0 && page < p.num_pages) z = page * p.h_kv + u.head;
                    else atomicCAS(p.err, 0u, (kTagTree << 16) | kSiteBadData | 1u);
                };
                // the next place of the ring, once it is free
                auto claim = [&]() -> bool { return warp_wait(bar(L::bEmpty) + 8u * stage, phase ^ 1u, wc, 1); };
                auto load = [&](const CUtensorMap *m, uint32_t full, int y, int z) {
                    if (loads)
                        tma_load_3d(sbase + L::kRing + stage * L::kTileBytes + col * L::kChunkBytes + mine * box * 128, m,
                                    full, col * (128 / L::kEb), y, z);
                    if (++stage == L::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                };
                const bool both = kPair && u.ntok > tpc;
                int y0, z0, y1, z1;  // of tiles i and i + 1
                place(0, y0, z0);
                place(1, y1, z1);
                auto alone = [&](int y, int z) {  // a unit's first K tiles have barriers to themselves
                    if (!(ok = claim())) return;
                    const uint32_t full = bar(L::bFull) + 8u * stage;
                    if (lane == 0) mbar_arrive_expect_tx(full, L::kTileBytes);
                    __syncwarp();
                    load(&tm_k, full, y, z);
                };
                alone(y0, z0);
                if (ok && !both && n > 1) alone(y1, z1);
                for (int i = 0; i < n && ok; ++i) {
                    int y2, z2;
                    place(i + 2, y2, z2);
                    const bool pair = i + (both ? 1 : 2) < n;
                    const uint32_t full = bar(L::bFull) + 8u * stage;
                    if (!(ok = claim())) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, pair ? 2 * L::kTileBytes : L::kTileBytes);
                    __syncwarp();
                    load(&tm_v, full, y0, z0);
                    if (pair) {
                        if (!(ok = claim())) break;
                        // its own barrier counts the use all the same
                        if (lane == 0) mbar_arrive(bar(L::bFull) + 8u * stage);
                        load(&tm_k, full, both ? y1 : y2, both ? z1 : z2);
                    }
                    y0 = y1;
                    z0 = z1;
                    y1 = y2;
                    z1 = z2;
                }
            }
            // every load issued must land before the CTA may exit
            for (int s = 0; s < L::kStages; ++s) {  // the phase that the place's last use completes, or the one before the first
                const uint32_t last = s < (int)stage ? phase : phase ^ 1u;
                mbar_wait_drain(bar(L::bFull + s), last);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ======================================================== products
            __syncthreads();
            {
                // The whole warp walks and waits, and one elected lane issues: so the compiler knows the
                // descriptors to be the warp's and not a lane's (one lane alone in this branch took 112 us
                // for 32 x 13 trees of E4M3, this 110; 24 x 36 with 8 heads a key/value head 168, 138).
                const bool issuer = elect_one();
                Units walk(p, *start);
                constexpr uint32_t idesc_s = kFp8 ? make_idesc_e4m3(kTileM, kTileN, false, false)
                                                  : make_idesc_f16(kTileM, kTileN, kBf16, false, false);
                // P's terms: E5M2, then E4M3
                constexpr uint32_t idesc_o = kFp8 ? make_idesc_e5m2_e4m3(kTileM, D, false, true)
                                                  : make_idesc_f16(kTileM, D, kBf16, false, true);
                constexpr uint32_t idesc_lo = make_idesc_e4m3(kTileM, D, false, true);
                constexpr uint32_t kChunk16 = L::kChunkBytes >> 4, kTile16 = L::kTileBytes >> 4;
                const uint64_t dQ = smem_desc_sw128(sbase + L::kQ, 16, 1024);
                const uint64_t dK = smem_desc_sw128(sbase + L::kRing, 16, 1024);
                const uint64_t dV = smem_desc_sw128(sbase + L::kRing, L::kChunkBytes, 1024);
                auto issue_s = [&](int x, int qx, uint32_t stage) {  // of Q tile qx
                    const uint64_t b = dK + stage * kTile16;
#pragma unroll
                    for (int term = 0; term < kQTerms; ++term) {
                        const uint64_t a = dQ + (qx * L::kQTerms + term) * kTile16;
#pragma unroll
                        for (int k = 0; k < D * L::kEb / 32; ++k) {
                            const uint32_t off = (k / 4) * kChunk16 + (k % 4) * 2;
                            if (!issuer) continue;
                            if constexpr (kFp8)
                                mma_ss_f8(tmem + L::kColS + x * 128, a + off, b + off, idesc_s, term > 0 || k > 0);
                            else
                                mma_ss(tmem + L::kColS + x * 128, a + off, b + off, idesc_s, k > 0);
                        }
                    }
                    if (issuer) mma_commit(bar(L::bSFull + x));
                };
                // P_x lies in S_x's columns; S_x of the chain's next tile is
                // issued behind P_x V, and one thread's products run in order
                auto issue_pv = [&](int x, uint32_t stage, bool acc) {
                    const uint64_t b = dV + stage * kTile16;
#pragma unroll
                    for (int term = 0; term < kPTerms; ++term)
#pragma unroll
                        for (int k = 0; k < kTileN * L::kEb / 32; ++k) {
                            const uint64_t v = b + k * ((4096 / L::kEb) >> 4);
                            const uint32_t o = tmem + L::kColO + x * D, pc = tmem + L::kColS + x * 128 + term * 32 + k * 8;
                            const uint32_t add = (acc || term > 0 || k > 0) ? 1u : 0u;
                            if (!issuer) continue;
                            if constexpr (kFp8) mma_ts_f8(o, pc, v, term == 0 ? idesc_o : idesc_lo, add);
                            else mma_ts(o, pc, v, idesc_o, add);
                        }
                };
                const int tpc = p.chain_tokens;
                int units = 0;
                uint32_t stage = 0, phase = 0;               // the ring's next place: tiles are used in the order they lie
                uint32_t p_phase[2] = {0, 0}, o_phase[2] = {1, 1};  // a first wait for O's release passes
                bool ok = true;
                auto full = [&](uint32_t site) { return mbar_wait(bar(L::bFull) + 8u * stage, phase, wc, site); };
                auto take = [&]() {
                    const uint32_t s = stage;
                    if (++stage == L::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    return s;
                };
                // One unit.  The loop is compiled apart for each of its two forms: this thread's own
                // instructions are what the products wait for when there are many rows.
                auto unit = [&](auto form, int n) {
                    constexpr bool both = decltype(form)::value;
                    constexpr int kAhead = both ? 1 : 2;  // the next S goes to the same chain; its K came with V
                    uint32_t k_stage = 0;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {  // first S of each chain
                        if (!both && x >= n) break;
                        if (!both || x == 0) {
                            if (!(ok = full(3))) return;
                            k_stage = take();
                        }
                        tc_fence_after();
                        issue_s(x, both ? x : 0, k_stage);
                    }
                    if (n <= kAhead && issuer) mma_commit(bar(L::bQEmpty));
                    uint32_t v_stage = 0;
                    // two steps a turn: both chains of one tile, or one tile of each chain
                    for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int i = both ? i0 : i0 + x;
                            if (i >= n) break;
                            const bool next = i + kAhead < n;
                            if (!both || x == 0) {
                                if (!(ok = full(5))) return;
                                v_stage = take();
                                if (next) k_stage = take();
                            }
                            if (!(ok = mbar_wait(bar(L::bPReady + x), p_phase[x], wc, 4))) return;
                            p_phase[x] ^= 1u;
                            if (i < kAhead) {
                                if (!(ok = mbar_wait(bar(L::bOFree + x), o_phase[x], wc, 6))) return;
                                o_phase[x] ^= 1u;
                            }
                            tc_fence_after();
                            issue_pv(x, v_stage, i >= kAhead);
                            if (!next) {
                                if (issuer) mma_commit(bar(L::bOFull + x));
                            } else {
                                issue_s(x, both ? x : 0, k_stage);
                                if (issuer && i + kAhead == n - 1 && (!both || x == 1)) mma_commit(bar(L::bQEmpty));  // the last reader of Q
                            }
                        }
                    }
                };
                while (ok && walk.next(u)) {
                    const int n = u.tb - u.ta;
                    if (!(ok = mbar_wait(bar(L::bQFull), units & 1, wc, 2))) break;
                    if (kPair && u.ntok > tpc) unit(std::integral_constant<bool, kPair>{}, n);
                    else unit(std::false_type{}, n);
                    ++units;
                }
                if (issuer) mma_commit(bar(L::bMmaIdle));
                mbar_wait_drain(bar(L::bMmaIdle), 0);
            }
            __syncwarp();
        } else {
            // ======================================================== Q
            const int tpc = p.chain_tokens;
            int units = 0;
            __syncthreads();
            Units walk(p, *start);
            if constexpr (!kFp8) {
                // boxes of 64 columns x group heads x the chain's tokens; rows behind the request's
                // tokens hold other tokens or zeros, and nobody reads their results
                if (warp == 2 && lane == 0) {
                    while (walk.next(u)) {
                        if (units > 0 && !mbar_wait(bar(L::bQEmpty), (units - 1) & 1, wc, 8)) break;
                        const int xs = kPair && u.ntok > tpc ? 2 : 1;
                        mbar_arrive_expect_tx(bar(L::bQFull), xs * kSplit * L::kChunks * tpc * p.group * 128);
                        for (int x = 0; x < xs; ++x)
#pragma unroll
                            for (int rep = 0; rep < kSplit; ++rep)
#pragma unroll
                                for (int c = 0; c < L::kChunks; ++c)
                                    tma_load_3d(sbase + L::kQ + x * L::kQBytes + c * L::kChunkBytes + rep * L::kUnique * 128,
                                                &tm_q, bar(L::bQFull), c * 64, u.head * p.group, u.q0 + u.tok + x * tpc);
                        ++units;
                    }
                    if (units > 0) mbar_wait_drain(bar(L::bQFull), (units - 1) & 1);
                }
                __syncwarp();
            } else {
                const int who = threadIdx.x - 64;  // 0..63
                float *qscale = reinterpret_cast<float *>(smem + L::kQScale);
                constexpr int kVecs = D / 8;   // 16-byte pieces of a row: a half warp reads one
                constexpr int kAhead = 8;      // pieces of a thread in flight
                bool ok = true;
                while (ok && walk.next(u)) {
                    for (int x = 0; x < (kPair && u.ntok > tpc ? 2 : 1) && ok; ++x) {
                        const int rows = min(u.ntok - x * tpc, tpc) * p.group;
                        const int64_t tok0 = u.q0 + u.tok + x * tpc;
                        for (int e0 = who; e0 - who < max(rows, 1) * kVecs; e0 += 64 * kAhead) {
                            uint4 raw[kAhead];
#pragma unroll
                            for (int a = 0; a < kAhead; ++a) {
                                const int e = e0 + a * 64, r = e / kVecs, v = e % kVecs;
                                raw[a] = make_uint4(0, 0, 0, 0);
                                if (r < rows)
                                    raw[a] = *reinterpret_cast<const uint4 *>(
                                        static_cast<const uint16_t *>(p.q) + (tok0 + r / p.group) * p.q_stride +
                                        (int64_t)(u.head * p.group + r % p.group) * D + v * 8);
                            }
                            // the first loads are under way while the unit before still reads Q
                            if (x == 0 && e0 == who && units > 0 &&
                                !(ok = warp_wait(bar(L::bQEmpty), (units - 1) & 1, wc, 8)))
                                break;
#pragma unroll
                            for (int a = 0; a < kAhead; ++a) {
                                const int e = e0 + a * 64, r = e / kVecs, v = e % kVecs;
                                const bool have = r < rows;
                                float f[8];
                                const uint32_t w[4] = {raw[a].x, raw[a].y, raw[a].z, raw[a].w};
                                float top = 0.f;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 t = unpack2<kBf16>(w[i]);
                                    f[2 * i] = t.x;
                                    f[2 * i + 1] = t.y;
                                    top = fmaxf(top, fmaxf(fabsf(t.x), fabsf(t.y)));
                                }
#pragma unroll
                                for (int off = kVecs / 2; off > 0; off >>= 1)
                                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                                // 2^(7 - e) takes the row's largest value, 2^e .. 2^(e+1), to 2^7 .. 2^8
                                const int ex = min(max((int)(__float_as_uint(top) >> 23), 10), 250);
                                const float up = __uint_as_float((uint32_t)(127 + 7 - (ex - 127)) << 23);
                                const float down = __uint_as_float((uint32_t)(127 - 7 + (ex - 127)) << 23);
                                if (have && v == 0) qscale[x * 128 + r] = down;
#pragma unroll
                                for (int i = 0; i < 8; ++i) f[i] *= up;
#pragma unroll
                                for (int term = 0; term < kQTerms; ++term) {
                                    const uint2 code = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]),
                                                                  pack_e4m3x4(f[4], f[5], f[6], f[7]));
                                    if (have) {
#pragma unroll
                                        for (int rep = 0; rep < kSplit; ++rep) {
                                            const int row = r + rep * L::kUnique;
                                            *reinterpret_cast<uint2 *>(smem + L::kQ + x * L::kQBytes + term * L::kTileBytes +
                                                                       row * 128 + (((v / 2) ^ (row & 7)) << 4) + (v & 1) * 8) = code;
                                        }
                                    }
                                    if (term + 1 < kQTerms) {
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            uint32_t h2;
                                            const uint16_t two = (uint16_t)((i < 2 ? code.x : code.y) >> (16 * (i & 1)));
                                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
                                            const float2 t = unpack2<false>(h2);
                                            f[2 * i] -= t.x;
                                            f[2 * i + 1] -= t.y;
                                        }
                                    }
                                }
                            }
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::bQFull));
                    ++units;
                }
            }
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ============================================================ softmax
        const int x = (warp - 4) >> 2;             // chain
        const int quad = warp & 3;
        const int ln = quad * 32 + lane;           // TMEM lane
        const int row = ln % L::kUnique;           // row of the chain's tile
        const int slice = quad * kSplit / 4;       // this repeat's keys: [slice kKeys, (slice + 1) kKeys)
        constexpr int kKeys = kTileN / kSplit;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t scol = t_lane + L::kColS + x * 128, ocol = t_lane + L::kColO + x * D;
        const int tpc = p.chain_tokens;
        const float *qscale = reinterpret_cast<const float *>(smem + L::kQScale);
        const float descale_v = kFp8 ? *p.descale_v : 1.f;
        const int tok_l = row / p.group;           // the row's token in the chain's tile
        // P is exp2(x - base).  base follows the running maximum with a lag of
        // up to kLag (log2), so O is seldom rescaled.  P is raised by 2^kRaise
        // so that small weights keep their bits: fp16 to at most 2^15, which
        // leaves weights off by up to 2^-32 of the row's largest and not
        // 2^-25 (30,000 keys of such a weight are a thousandth of O); an E4M3
        // cache's terms up to 2^11.5, whose rest of at most 2^8 still is an
        // E4M3 value; bf16 has fp32's exponents
        constexpr float kRaise = kFp8 ? 8.f : kBf16 ? 0.f : 7.f, kLag = kFp8 ? 3.5f : 8.f;
        int it = 0, units = 0, cnt = 0, uo0 = 0, uo1 = 0, joins = 0;
        bool ok = true;
        __syncthreads();
        Units walk(p, *start);
        while (ok && walk.next(u)) {
            const int n = u.tb - u.ta;
            const bool both = kPair && u.ntok > tpc;  // the chains' rows are different ones
            const int xr = both ? x : 0;              // the chain's rows: tile of Q, part of the unit
            float sl2 = p.scale_log2;
            if constexpr (kFp8) {
                if (!(ok = warp_wait(bar(L::bQFull), units & 1, wc, 9))) break;
                sl2 *= *p.descale_k * qscale[xr * 128 + row];
                if (sl2 == 0.f) sl2 = 1.17549435e-38f;  // a row of zeros: masked scores stay -inf and not NaN
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::bQEmpty));
            }
            const bool row_ok = tok_l < min(u.ntok - xr * tpc, tpc);
            const int tok = u.tok + xr * tpc + tok_l;  // token of the request
            float base = -INFINITY;  // exponent base, kRaise below the maximum it followed
            float l = 0.f;           // sum of P
            bool some = false;       // O_x holds something
            const bool releases = quad == 0 && (!both || x == 1);
            const int step = both ? 1 : 2;
            const int last = both || ((n - 1) & 1) == x ? n - 1 : n - 2;  // the chain's last tile
            {
                for (int i = both ? 0 : x; i < n; i += step, ++cnt) {
                    const int k0 = (u.ta + i) * kTileN;
                    const bool edge = k0 + kTileN > min(u.ctx, u.end);  // keys that not every row sees
                    uint32_t seen[kKeys / 32];
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < kKeys / 32; ++c)
                            seen[c] = row_ok ? seen_bits(p, u, tok, k0 + slice * kKeys + c * 32) : 0u;
                    }
                    uint32_t live = 0xffffffffu;  // of keys k0 + 32 quad ..: those that some row of the unit sees
                    if (edge) {
                        if (p.mask) {
                            live = 0u;
                            for (int t = lane; t < u.ntok; t += 32) live |= seen_bits(p, u, u.tok + t, k0 + quad * 32);
                            live = __reduce_or_sync(0xffffffffu, live);
                        } else {
                            const int have = u.end - (k0 + quad * 32);
                            live = have >= 32 ? 0xffffffffu : have <= 0 ? 0u : (1u << have) - 1u;
                        }
                    }
                    if (!(ok = warp_wait(bar(L::bSFull + x), cnt & 1, wc, 10))) break;
                    tc_fence_after();
                    // S_x is done, and the chain's P V before it: their tiles' places are free (the
                    // issuing thread, which every commit would hold up, leaves this to the softmax)
                    if (releases && lane == 0) {
                        mbar_arrive(bar(L::bEmpty + (it + k_pos(both, i)) % L::kStages));
                        if (some) mbar_arrive(bar(L::bEmpty + (it + v_pos(both, i - step, n)) % L::kStages));
                    }
                    uint32_t s[kKeys];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(scol + slice * kKeys + c * 32, s + c * 32);
                    tmem_ld_wait_regs<kKeys>(s);
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if (!(seen[c / 32] >> (c % 32) & 1u)) s[c] = __float_as_uint(-INFINITY);
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kKeys; c += 8) {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            mx4[v] = fmax3(mx4[v], __uint_as_float(s[c + 2 * v]), __uint_as_float(s[c + 2 * v + 1]));
                    }
                    const float m_tile = fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3])) * sl2 - kRaise;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (m_tile > base + kLag) {
                        rescale = true;
                        alpha = ex2_approx(base - m_tile);
                        base = m_tile;
                        l *= alpha;
                    }
                    const float b = base == -INFINITY ? 0.f : base;
                    const uint64_t sl2_2 = f2_pack(sl2, sl2), nb_2 = f2_pack(-b, -b);
                    uint64_t sum2[4] = {0, 0, 0, 0};
                    constexpr uint32_t kZero[32] = {};
                    if constexpr (!kFp8) {
#pragma unroll
                        for (int c = 0; c < kKeys / 2; ++c) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2_2, nb_2), x0, x1);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            sum2[c & 3] = f2_add(sum2[c & 3], f2_pack(p0, p1));
                            s[c] = pack2<kBf16>(p0, p1);
                        }
                        if constexpr (kSplit == 1) {
                            tmem_st32(scol, s);
                            tmem_st32(scol + 32, s + 32);
                        } else if constexpr (kSplit == 2) {
                            tmem_st32(scol + slice * 32, s);
                            tmem_st32(scol + (slice ^ 1) * 32, kZero);
                        } else {
#pragma unroll
                            for (int c = 1; c < 4; ++c) tmem_st16(scol + (slice ^ c) * 16, kZero);
                            tmem_st16(scol + slice * 16, s);
                        }
                    } else {
                        uint32_t t1[kKeys / 4], t2[kKeys / 4], t3[kPTerms > 2 ? kKeys / 4 : 1];
#pragma unroll
                        for (int c = 0; c < kKeys / 4; ++c) {
                            uint32_t h[2], up[2];
                            uint16_t lo[2], lo2[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float x0, x1;
                                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[4 * c + 2 * e]), __uint_as_float(s[4 * c + 2 * e + 1])),
                                                 sl2_2, nb_2), x0, x1);
                                const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                                sum2[(2 * c + e) & 3] = f2_add(sum2[(2 * c + e) & 3], f2_pack(p0, p1));
                                h[e] = pack2<false>(p0, p1);
                                // an fp16 value's high byte is an E5M2 value: rounded by half of what
                                // the byte below is worth; what that leaves goes to E4M3
                                up[e] = h[e] + 0x00800080u;
                                uint32_t rest;
                                asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h[e]), "r"(up[e] & 0xff00ff00u));
                                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo[e]) : "r"(rest));
                                if constexpr (kPTerms > 2)  // and of that the rest to a second E4M3
                                    asm("{\n\t.reg .b32 l;\n\tcvt.rn.f16x2.e4m3x2 l, %1;\n\tsub.rn.f16x2 l, %2, l;\n\t"
                                        "cvt.rn.satfinite.e4m3x2.f16x2 %0, l;\n\t}"
                                        : "=h"(lo2[e]) : "h"(lo[e]), "r"(rest));
                            }
                            t1[c] = __byte_perm(up[0], up[1], 0x7531);
                            t2[c] = (uint32_t)lo[0] | ((uint32_t)lo[1] << 16);
                            if constexpr (kPTerms > 2) t3[c] = (uint32_t)lo2[0] | ((uint32_t)lo2[1] << 16);
                        }
                        auto put = [&](uint32_t col, const uint32_t *t) {
                            if constexpr (kSplit == 1) {
                                tmem_st32(col, t);
                            } else if constexpr (kSplit == 2) {
                                tmem_st16(col + slice * 16, t);
                                tmem_st16(col + (slice ^ 1) * 16, kZero);
                            } else {
                                tmem_st8(col + slice * 8, t);
#pragma unroll
                                for (int c = 1; c < 4; ++c) tmem_st8(col + (slice ^ c) * 8, kZero);
                            }
                        };
                        put(scol, t1);
                        put(scol + 32, t2);
                        if constexpr (kPTerms > 2) put(scol + 64, t3);
                    }
                    {
                        float a0, a1;
                        f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), a0, a1);
                        l += a0 + a1;
                    }
                    if (some && __any_sync(0xffffffffu, rescale)) {
                        // S_x's commit followed every earlier product, so O_x is at rest
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(ocol + c * 32, o);
                            tmem_ld_wait_regs<32>(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(ocol + c * 32, o);
                        }
                    }
                    some = true;
                    if (edge && live != 0xffffffffu) {
                        // a value that no row weighs may be anything: 0 x NaN must not enter the product
                        const int pos = it + v_pos(both, i, n), st = pos % L::kStages;
                        if (!(ok = warp_wait(bar(L::bFull + st), (pos / L::kStages) & 1, wc, 11))) break;
                        if (!(live >> lane & 1u)) {
                            uint4 *v = reinterpret_cast<uint4 *>(smem + L::kRing + st * L::kTileBytes + ln * 128);
#pragma unroll
                            for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[c * (L::kChunkBytes / 16) + e] = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::bPReady + x));
                }
                if (!ok) break;
            }
            // ---- the unit's rows are done as far as this CTA runs them
            const bool whole = u.ta == 0 && u.tb == u.unit_tiles;
            float *part = parts + (2 * (int64_t)blockIdx.x + (u.ta > 0 ? 0 : 1)) * L::kPartFloats;
            float2 *part_ml = reinterpret_cast<float2 *>(part + (size_t)kRows * D);
            const int part_row = xr * 128 + row;
            const int64_t out_row = (int64_t)(u.q0 + tok) * p.h + u.head * p.group + row - tok_l * p.group;
            auto sync = [&]() -> bool {  // all eight warps, bounded
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::bJoin));
                const bool y = warp_wait(bar(L::bJoin), joins & 1, wc, 13);
                ++joins;
                return y;
            };
            if (both) {
                if (!(ok = warp_wait(bar(L::bOFull + x), (x ? uo1 : uo0) & 1, wc, 12))) break;
                ++uo0;
                ++uo1;
                tc_fence_after();
                if (releases && lane == 0) mbar_arrive(bar(L::bEmpty + (it + v_pos(both, last, n)) % L::kStages));
                const float f = whole ? (l > 0.f ? descale_v / l : 0.f) : 1.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(ocol + c * 32, o);
                    tmem_ld_wait_regs<32>(o);
                    if (c == D / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {  // four warps read this chain's O: two arrivals each
                            mbar_arrive(bar(L::bOFree + x));
                            mbar_arrive(bar(L::bOFree + x));
                        }
                    }
                    if (!row_ok) continue;
                    if (whole) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack2<kBf16>(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                        uint8_t *dst = static_cast<uint8_t *>(p.o) + (out_row * D + c * 32) * 2;
                        st_global_32b(dst, pk);
                        st_global_32b(dst + 32, pk + 8);
                    } else {
                        uint8_t *dst = reinterpret_cast<uint8_t *>(part + (size_t)part_row * D + c * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) st_global_32b(dst + e * 32, o + 8 * e);
                    }
                }
                if (row_ok) {
                    if (!whole) part_ml[part_row] = make_float2(base, l);
                    else if (p.lse) p.lse[out_row] = l > 0.f ? (base + lg2_approx(l)) * kLn2 : -INFINITY;
                }
            } else {
                // Join the two chains and the repeats of every row.  Both chains' O of a row lie in the
                // same TMEM lane, so a warp adds them by itself: warps of chain 0 take the first half of
                // the columns, those of chain 1 the second; repeats go through shared memory, each warp
                // keeping kOwn of its columns and giving the rest to the warps that keep those.
                // A chain without a tile in the next unit gets to its write of `stats` there without
                // waiting for the other chain's warps, which may have to read this unit's sums still.
                // Repeats meet again further down; without them the warps arrive once more behind
                // their reads, and wait for that arrival before they write the next unit's sums.
                float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
                if (kSplit == 1 && joins > 0 && !(ok = warp_wait(bar(L::bJoin), (joins - 1) & 1, wc, 14))) break;
                stats[x * 128 + ln] = make_float2(base, l);
                if (!(ok = sync())) break;
                float top = -INFINITY, all = 0.f, f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int rep = 0; rep < kSplit; ++rep) {
                        const float2 v = stats[y * 128 + rep * L::kUnique + row];
                        if (v.y > 0.f) top = fmaxf(top, v.x);
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int rep = 0; rep < kSplit; ++rep) {
                        const float2 v = stats[y * 128 + rep * L::kUnique + row];
                        if (v.y > 0.f) all += ex2_approx(v.x - top) * v.y;
                    }
                    const float2 v = stats[y * 128 + ln];
                    f[y] = v.y > 0.f ? ex2_approx(v.x - top) : 0.f;
                }
                if constexpr (kSplit == 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::bJoin));
                    ++joins;
                }
                const bool two = n > 1;  // chain 1 has a tile
                ok = warp_wait(bar(L::bOFull + 0), uo0 & 1, wc, 12) &&
                     (!two || warp_wait(bar(L::bOFull + 1), uo1 & 1, wc, 12));
                if (!ok) break;
                ++uo0;
                uo1 += two ? 1 : 0;
                tc_fence_after();
                if (some && releases && lane == 0) mbar_arrive(bar(L::bEmpty + (it + v_pos(both, last, n)) % L::kStages));
                const float scale = whole ? (all > 0.f ? descale_v / all : 0.f) : 1.f;
                f[0] *= scale;
                f[1] *= scale;
                constexpr int kOwn = L::kOwn, kHalf = D / 2;
                float *join = reinterpret_cast<float *>(smem + L::kJoin);
                // floats that repeat `from` gives to the warp of quadrant q of this half, kGive at a time
                constexpr int kGive = L::kGive;
                auto given = [&](int q, int from) {
                    const int to = q * kSplit / 4, at = from < to ? from : from - 1;
                    return join + (((x * 4 + q) * (kSplit - 1) + at) * 32 + lane) * kGive;
                };
                const int turn = lane * kGive / 32;  // keeps lanes of one bank apart
                uint8_t *dst = whole ? static_cast<uint8_t *>(p.o) + (out_row * D + x * kHalf + slice * kOwn) * 2
                                     : reinterpret_cast<uint8_t *>(part + (size_t)row * D + x * kHalf + slice * kOwn);
                auto put = [&](const float *v, int at) {  // 16 columns of the row, or 8
                    constexpr int kCols = kOwn < 16 ? kOwn : 16;
                    if (whole) {
                        uint32_t pk[kCols / 2];
#pragma unroll
                        for (int e = 0; e < kCols / 2; ++e) pk[e] = pack2<kBf16>(v[2 * e], v[2 * e + 1]);
                        if constexpr (kCols == 16) st_global_32b(dst + at * 2, pk);
                        else *reinterpret_cast<uint4 *>(dst + at * 2) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < kCols; e += 8)
                            st_global_32b(dst + (at + e) * 4, reinterpret_cast<const uint32_t *>(v + e));
                    }
                };
                float v[kSplit == 1 ? 32 : kHalf];  // without repeats 32 columns go out at a time
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    uint32_t o[32], o1[32];
                    tmem_ld32(t_lane + L::kColO + x * kHalf + c, o);
                    if (two) tmem_ld32(t_lane + L::kColO + D + x * kHalf + c, o1);
                    tmem_ld_wait_regs<32>(o);
                    if (two) tmem_ld_wait_regs<32>(o1);
                    if (c + 32 == kHalf) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(L::bOFree + 0));
                            if (two) mbar_arrive(bar(L::bOFree + 1));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int at = (kSplit == 1 ? 0 : c) + e;
                        v[at] = __uint_as_float(o[e]) * f[0];
                        if (two) v[at] += __uint_as_float(o1[e]) * f[1];
                    }
                    if (kSplit == 1 && row_ok) {
                        put(v, c);
                        put(v + 16, c + 16);
                    }
                }
                if constexpr (kSplit > 1) {
                    float own[kOwn];
#pragma unroll
                    for (int r = 0; r < kOwn; r += kGive) {
                        if (r > 0 && !(ok = sync())) break;  // the columns before have been read
#pragma unroll
                        for (int to = 0; to < kSplit; ++to) {  // the repeat that keeps columns [to kOwn, (to + 1) kOwn)
                            if (to == slice) {
#pragma unroll
                                for (int e = 0; e < kGive; ++e) own[r + e] = v[to * kOwn + r + e];
                            } else {
                                float *g = given(kSplit == 4 ? to : to * 2 + (quad & 1), slice);
#pragma unroll
                                for (int e = 0; e < kGive; ++e) g[e ^ turn] = v[to * kOwn + r + e];
                            }
                        }
                        if (!(ok = sync())) break;
#pragma unroll
                        for (int from = 0; from < kSplit; ++from) {
                            if (from == slice) continue;
                            const float *g = given(quad, from);
#pragma unroll
                            for (int e = 0; e < kGive; ++e) own[r + e] += g[e ^ turn];
                        }
                    }
                    if (!ok) break;
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < kOwn; e += 16) put(own + e, e);
                    }
                }
                if (row_ok && x == 0 && slice == 0) {
                    if (!whole) part_ml[row] = make_float2(top, all);
                    else if (p.lse) p.lse[out_row] = all > 0.f ? (top + lg2_approx(all)) * kLn2 : -INFINITY;
                }
            }
            it += 2 * n;
            ++units;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the parts of the units that were cut: that of the CTA before the first
// to continue the unit and those of the ones that continue it, in that order.
// A record of each continuing CTA names its unit, and the CTAs here that read
// them take the unit's rows in turn, so that the grid grows with the rows of
// all cut units and not with rows times CTAs (a 6 x 42 tree of 126 rows, 12
// units in 150 parts: the pair of kernels takes 15.0 us and not 22.2).  One
// warp a row and group of parts: kAhead parts' statistics and rows are read at
// once and added under the running maximum.  The code is short on purpose: it
// runs for a few microseconds, and its first pass through an instruction is a
// miss.  Where units are few, and so have many parts, kWarps warps share a
// row's (four: 15.0 us on the same tree, eight: 17.1).
template <int D, int kEl, bool kFp8, int kRows, int kWarps>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p) {
    constexpr size_t kPart = (size_t)kRows * (D + 2);
    constexpr int kPer = D / 32, kAhead = kWarps == 1 ? 2 : 4;
    using Vec = std::conditional_t<kPer == 4, float4, float2>;
    __shared__ float s_acc[8][D];
    __shared__ float2 s_ml[8];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Cut cut = reinterpret_cast<const Cut *>(p.workspace)[blockIdx.x + 1];
    if (cut.parts == 0) return;
    const int c = blockIdx.x + 1 - cut.mine, sharers = cut.parts - 1;
    const int rows = p.chain_tokens * p.group;  // of a chain
    const int end = cut.ntok * p.group;
    const float *parts = reinterpret_cast<const float *>(p.workspace + kTreeMaxCtas * sizeof(Cut));
    const float descale = kFp8 ? *p.descale_v : 1.f;
#pragma unroll 1
    for (int at0 = (blockIdx.y * sharers + cut.mine) * (8 / kWarps); at0 < end; at0 += gridDim.y * sharers * (8 / kWarps)) {
        const int at = at0 + warp / kWarps;           // row of the unit
        const int row = at / rows * 128 + at % rows;  // in a part
        float top = -INFINITY, sum = 0.f, acc[kPer] = {};
#pragma unroll 1
        for (int i0 = warp % kWarps * kAhead; at < end && i0 < cut.parts; i0 += kWarps * kAhead) {
            float2 v[kAhead];
            Vec o[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int i = min(i0 + a, cut.parts - 1);
                const float *part = parts + (i == 0 ? 2 * (int64_t)(c - 1) + 1 : 2 * (int64_t)(c - 1 + i)) * kPart;
                v[a] = reinterpret_cast<const float2 *>(part + (size_t)kRows * D)[row];
                o[a] = reinterpret_cast<const Vec *>(part + (size_t)row * D)[lane];
                if (i0 + a >= cut.parts || !(v[a].y > 0.f)) v[a] = make_float2(-INFINITY, 0.f);
            }
            float now = top;
#pragma unroll
            for (int a = 0; a < kAhead; ++a) now = fmaxf(now, v[a].x);
            const float base = now == -INFINITY ? 0.f : now, old = ex2_approx(top - base);
            top = now;
            sum *= old;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= old;
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const float f = ex2_approx(v[a].x - base);
                sum += f * v[a].y;
                const float *w = reinterpret_cast<const float *>(&o[a]);
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] += f > 0.f ? f * w[e] : 0.f;
            }
        }
        if constexpr (kWarps > 1) {
            if (lane == 0) s_ml[warp] = make_float2(top, sum);
#pragma unroll
            for (int e = 0; e < kPer; ++e) s_acc[warp][lane * kPer + e] = acc[e];
            __syncthreads();
#pragma unroll 1
            for (int w = 1; w < kWarps && warp % kWarps == 0; ++w) {
                const float2 v = s_ml[warp + w];
                const float now = fmaxf(top, v.x), base = now == -INFINITY ? 0.f : now;
                const float old = ex2_approx(top - base), f = ex2_approx(v.x - base);
                top = now;
                sum = sum * old + f * v.y;
#pragma unroll
                for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * old + f * s_acc[warp + w][lane * kPer + e];
            }
        }
        if (kWarps > 1) __syncthreads();  // the next row's sums go to the same place
        if (warp % kWarps != 0 || at >= end) continue;
        const float inv = sum > 0.f ? descale / sum : 0.f;
        const int64_t out = (int64_t)(cut.q_tok + at / p.group) * p.h + cut.head * p.group + at % p.group;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + out * D + lane * kPer);
#pragma unroll
        for (int e = 0; e < kPer; e += 2) dst[e / 2] = pack2<kEl == kElBf16>(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0 && p.lse) p.lse[out] = sum > 0.f ? (top + lg2_approx(sum)) * kLn2 : -INFINITY;
    }
}

template <int D, int kEl, bool kFp8, int kRows>
cudaError_t launch_rows(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p, int max_q, int grid,
                        cudaStream_t stream, const KernelTimer &timer) {
    using L = TreeLayout<D, kFp8, kRows>;
    auto kern = tree_kernel<D, kEl, kFp8, kRows>;
    // setmaxnreg.inc waits for registers that the launch must have: a build
    // with another count is not launched
    static std::atomic<int> launch_regs{0};
    int regs = launch_regs.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes fa{};
        const cudaError_t q = cudaFuncGetAttributes(&fa, kern);
        if (q != cudaSuccess) return q;
        regs = fa.numRegs;
        launch_regs.store(regs, std::memory_order_relaxed);
    }
    if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != cudaSuccess) return e;
    if (timer.start) cudaEventRecord(timer.start, stream);
    e = launch_overlapped(kern, dim3(grid), dim3(kThreads), L::kBytes, stream, tq, tk, tv, p);
    // units of one key tile cannot be cut, nor can one CTA's
    if (e == cudaSuccess && grid > 1 && p.max_kv > kTileN) {
        const int tpt = tokens_per_tile<kRows>(p);
        const int rows = std::min(max_q, tpt) * p.group;  // of a unit, at most
        const int64_t units = (int64_t)std::max(p.num_seqs, p.total_q / tpt) * p.h_kv;
        // Ragged requests share less well than this estimate and a second turn of a CTA costs 2 to 5
        // us, an idle CTA next to nothing: four times the CTAs that would do (one tree of 8 rows: 10.1
        // us; twice: 11.8; once: 15.0).
        const int64_t sharers = std::max(grid / units - 1, (int64_t)1);
        if (units * 4 <= grid) {  // about four parts a unit and more
            const int64_t turns = std::min<int64_t>((rows + 1) / 2, (2 * rows + sharers - 1) / sharers);
            e = launch_overlapped(tree_join_kernel<D, kEl, kFp8, kRows, 4>, dim3(grid - 1, turns), dim3(256), 0, stream, p);
        } else {
            e = launch_overlapped(tree_join_kernel<D, kEl, kFp8, kRows, 1>, dim3(grid - 1, (rows + 7) / 8), dim3(256), 0, stream,
                                  p);
        }
    }
    if (timer.stop) cudaEventRecord(timer.stop, stream);
    return e;
}

template <int D, int kEl, bool kFp8>
cudaError_t launch_type(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p, int max_q, int rows, int grid,
                        cudaStream_t stream, const KernelTimer &timer) {
    if (rows == 32) return launch_rows<D, kEl, kFp8, 32>(tq, tk, tv, p, max_q, grid, stream, timer);
    if (rows == 64) return launch_rows<D, kEl, kFp8, 64>(tq, tk, tv, p, max_q, grid, stream, timer);
    return launch_rows<D, kEl, kFp8, 256>(tq, tk, tv, p, max_q, grid, stream, timer);
}

}  // namespace

int tree_rows(int max_q, int group) {
    const int64_t rows = (int64_t)max_q * group;
    return rows <= 32 ? 32 : rows <= 64 ? 64 : 256;
}

// Bounds of the units there can be, and of the places of their list.
static int64_t tree_units(int max_q, int total_q, int num_seqs, int h_kv, int group) {
    const int rows = tree_rows(max_q, group);
    const int tokens = (rows == 256 ? 2 : 1) * ((rows == 256 ? 128 : rows) / group);
    return ((int64_t)total_q / tokens + num_seqs) * h_kv;
}
static int64_t tree_tiles(int max_kv) { return ((int64_t)max_kv + kTileN - 1) / kTileN + 1; }  // of a unit
int64_t tree_places(int max_q, int total_q, int num_seqs, int h_kv, int group, int max_kv) {
    const int64_t units = tree_units(max_q, total_q, num_seqs, h_kv, group), tiles = tree_tiles(max_kv);
    return units > INT32_MAX ? units : units * (2 * tiles + 8);
}

int tree_q_tokens(int max_q, int group) { return std::min(tree_rows(max_q, group), 128) / group; }

size_t tree_workspace_bytes(int max_q, int group, int d) {
    return kTreeMaxCtas * (sizeof(Cut) + 2 * (size_t)tree_rows(max_q, group) * (d + 2) * 4);
}

cudaError_t launch_tree_fwd(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p, int max_q, int dtype,
                            int cache_dtype, int sm_count, cudaStream_t stream, const KernelTimer &timer) {
    const int rows = tree_rows(max_q, p.group);
    // no more CTAs than key tiles there can be
    const int64_t tiles = tree_units(max_q, p.total_q, p.num_seqs, p.h_kv, p.group) * tree_tiles(p.max_kv);
    const int grid = (int)(tiles < sm_count ? tiles : sm_count < kTreeMaxCtas ? sm_count : kTreeMaxCtas);
#define SDPA_TREE_CASE(D_, EL_, FP8_)                                  \
    if (p.d == D_ && dtype == EL_ && (cache_dtype == kElE4m3) == FP8_) \
        return launch_type<D_, EL_, FP8_>(tq, tk, tv, p, max_q, rows, grid, stream, timer);
    SDPA_TREE_CASE(64, kElBf16, false)
    SDPA_TREE_CASE(64, kElFp16, false)
    SDPA_TREE_CASE(128, kElBf16, false)
    SDPA_TREE_CASE(128, kElFp16, false)
    SDPA_TREE_CASE(128, kElBf16, true)
    SDPA_TREE_CASE(128, kElFp16, true)
#undef SDPA_TREE_CASE
    return cudaErrorInvalidValue;
}

}  // namespace sdpa
