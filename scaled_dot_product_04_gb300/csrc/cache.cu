// Paged key/value cache: the plan of a step from its request lengths, the
// write of new keys and values to their slots, and the move of a verified
// tree's accepted path to the tree's front.
//
// Caches are [num_pages, h_kv, page_size, d]: one (page, head) is page_size
// contiguous rows, which is what the attention's tile loads want.  Request b
// owns the pages in row b of the block table; token t of it lives in page
// table[b][t / page_size] at offset t % page_size, and its slot is
// page * page_size + offset.
#include "cache.cuh"
#include "ptx.cuh"

namespace sdpa {
namespace {

SDPA_DEV void report_bad_data(uint32_t *err, uint32_t tag, uint32_t site) {
    atomicCAS(err, 0u, (tag << 16) | kSiteBadData | site);
}

// ------------------------------------------------------------------ plan
// Every CTA scans all requests itself (a chunk of them per thread), so one
// launch needs no pass of its own for the prefix sums and no CTA waits for
// another; then the first CTAs take the table rows, the others the tokens.
// It moves 8 bytes a token and is bound by its dependent reads (lengths, the
// token's request, its page): 32 requests with trees of 16 take 3.4 us, 1024
// prompts of 520,000 tokens in all 7.1 us, launch and host included.
constexpr int kPlanThreads = 256, kPlanTokens = 8;

// Sum of non-negative counts that stays at `cap` once it gets there (pages given back: at the
// pages there are, whatever the requests claim to hold).
SDPA_DEV int sat_add(int a, int b, int cap) { return a > cap - b ? cap : a + b; }

struct Request {
    int ctx, n, held, want, back, over;  // want: pages to take; back: to give back; over: refused by the table's width
};
SDPA_DEV Request load_request(const PlanParams &p, int b) {
    Request r;
    r.ctx = min(max(p.ctx[b], 0), INT32_MAX - p.max_new);
    const int n = p.fresh[b];
    r.held = min(max(p.held_in[b], 0), p.max_blocks);
    const bool done = n < 0;
    r.n = min(max(n, 0), p.max_new);
    const uint32_t len = (uint32_t)r.ctx + (uint32_t)r.n;  // at most 2^31 - 1
    const int need = (int)((len + (uint32_t)p.page_size - 1u) / (uint32_t)p.page_size);
    const int fit = min(need, p.max_blocks);
    r.want = done ? 0 : max(fit - r.held, 0);
    r.over = done ? 0 : need - fit;
    r.back = done ? r.held : 0;
    return r;
}

// Mask row of node i of the request whose tokens begin at `first`; its number
// of ancestors.  A parent is below its node, so the walk up visits the row's
// words from high to low.
SDPA_DEV int plan_node(const PlanParams &p, int t, int first, int i) {
    uint32_t *words = p.mask ? p.mask + (int64_t)t * p.mask_words : nullptr;
    const int have = p.mask ? p.mask_words : 0;
    int node = i, depth = 0, word = i >> 5;
    bool padding = false;
    uint32_t bits = 0u;
    for (int x = word + 1; x < have; ++x) words[x] = 0u;
    while (true) {
        const int x = node >> 5;
        if (x != word) {
            if (word < have) words[word] = bits;
            for (int y = x + 1; y < min(word, have); ++y) words[y] = 0u;
            word = x;
            bits = 0u;
        }
        bits |= 1u << (node & 31);
        const int up = p.parents[first + node];
        if (up == -1) break;
        if (up < -1 || up >= node) {
            padding = true;
            break;
        }
        node = up;
        ++depth;
    }
    if (word < have) words[word] = bits;
    for (int y = 0; y < min(word, have); ++y) words[y] = 0u;
    if (padding)
        for (int y = 0; y < have; ++y) words[y] = 0u;
    return padding ? 0 : depth;
}

// kTree: with parents.  A token's work is a few dependent loads, so without
// them a thread takes eight tokens (four: 7.7 us for 1024 prompts, eight 7.1) and
// writes 16 bytes at a time; with them the walks are the longest part and every
// token has a thread.
template <bool kTree>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p, int row_ctas) {
    constexpr int kPer = kTree ? 1 : kPlanTokens;
    const bool vectors = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
    __shared__ int s_n[kPlanThreads + 1], s_w[kPlanThreads + 1], s_b[kPlanThreads + 1];
    __shared__ int s_warp[4][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();  // nothing is read or written before the kernel ahead has ended
    const int per = (p.b + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(p.b, tid * per), r1 = min(p.b, r0 + per);
    int n = 0, w = 0, back = 0, over = 0;
    for (int r = r0; r < r1; ++r) {
        const Request q = load_request(p, r);
        n = sat_add(n, q.n, p.max_new);
        w += q.want;
        back = sat_add(back, q.back, p.num_pages);
        over = sat_add(over, q.over, INT32_MAX);
    }
    // inclusive scans of n, w and back over the warp, then over the warps
    int in = n, iw = w, ib = back;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, in, off), c = __shfl_up_sync(0xffffffffu, iw, off),
                  e = __shfl_up_sync(0xffffffffu, ib, off), f = __shfl_xor_sync(0xffffffffu, over, off);
        if (lane >= off) {
            in = sat_add(in, a, p.max_new);
            iw += c;
            ib = sat_add(ib, e, p.num_pages);
        }
        over = sat_add(over, f, INT32_MAX);
    }
    if (lane == 31) {
        s_warp[0][warp] = in;
        s_warp[1][warp] = iw;
        s_warp[2][warp] = ib;
        s_warp[3][warp] = over;
    }
    __syncthreads();
    int bn = 0, bw = 0, bb = 0;
    for (int i = 0; i < warp; ++i) {
        bn = sat_add(bn, s_warp[0][i], p.max_new);
        bw += s_warp[1][i];
        bb = sat_add(bb, s_warp[2][i], p.num_pages);
    }
    s_n[tid + 1] = sat_add(bn, in, p.max_new);
    s_w[tid + 1] = bw + iw;
    s_b[tid + 1] = sat_add(bb, ib, p.num_pages);
    if (tid == 0) s_n[0] = s_w[0] = s_b[0] = 0;
    __syncthreads();
    const int total = s_n[kPlanThreads], wanted = s_w[kPlanThreads], returned = s_b[kPlanThreads];
    const int pages = p.num_pages;
    const int head = min(max(p.ring_in[0], 0), max(pages - 1, 0));
    const int count = min(max(p.ring_in[1], 0), pages);
    auto ring_at = [&](int k) {  // entry k <= num_pages places behind the first free one (31 bits hold both)
        const int at = head + k;
        return at >= pages ? at - pages : at;
    };

    // the first row_ctas CTAs write the per-request outputs and table rows, a warp a request
    const int warps = row_ctas * (kPlanThreads / 32);
    for (int r = blockIdx.x * (kPlanThreads / 32) + warp; (int)blockIdx.x < row_ctas && r < p.b; r += warps) {
        const int c = r / per;
        int first_n = s_n[c], first_w = s_w[c], first_b = s_b[c];
        for (int i = c * per; i < r; ++i) {
            const Request q = load_request(p, i);
            first_n = sat_add(first_n, q.n, p.max_new);
            first_w += q.want;
            first_b = sat_add(first_b, q.back, pages);
        }
        const Request q = load_request(p, r);
        const int granted = min(max(count - first_w, 0), q.want);
        const int end_n = sat_add(first_n, q.n, p.max_new);
        int32_t *row = p.table + (int64_t)r * p.max_blocks;
        if (lane == 0) {
            if (r == 0) p.cu_new[0] = 0;
            p.cu_new[r + 1] = end_n;
            p.kv_lens[r] = p.fresh[r] < 0 ? 0 : q.ctx + (end_n - first_n);
            p.held_out[r] = q.back > 0 || p.fresh[r] < 0 ? 0 : q.held + granted;
        }
        for (int j = lane; j < q.want; j += 32)
            row[q.held + j] = j < granted ? p.free_ring[ring_at(first_w + j)] : -1;
        // pages given back go behind the free entries that were there, as far as the ring has room
        for (int j = lane; j < q.back; j += 32)
            if (count + first_b + j < pages) p.free_ring[ring_at(count + first_b + j)] = row[j];
    }
    if (blockIdx.x == 0 && tid == 0) {
        const int taken = min(wanted, count);
        if (p.b == 0) p.cu_new[0] = 0;
        p.ring_out[0] = pages > 0 ? ring_at(taken) : 0;
        p.ring_out[1] = min(count - taken + returned, pages);
        int over_all = 0;
        for (int i = 0; i < kPlanThreads / 32; ++i) over_all = sat_add(over_all, s_warp[3][i], INT32_MAX);
        p.ring_out[2] = sat_add(over_all, wanted - taken, INT32_MAX);
    }

    // the others the per-token outputs: kPer tokens in a row a thread, found by one search
    const int token_ctas = gridDim.x - row_ctas;
    for (int t0 = ((int)blockIdx.x - row_ctas) * kPlanThreads * kPer + tid * kPer; (int)blockIdx.x >= row_ctas && t0 < p.max_new;
         t0 += token_ctas * kPlanThreads * kPer) {
        int slot[kPer], position[kPer];
        int lo = 0, hi = kPlanThreads;  // s_n[lo] <= t0 < s_n[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_n[mid] <= t0) lo = mid;
            else hi = mid;
        }
        int r = lo * per, first = s_n[lo], first_w = s_w[lo];
        Request q{};
        if (t0 < total) q = load_request(p, r);
        int page = -1, page_blk = -1, page_row = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int t = t0 + e;
            slot[e] = -1;
            position[e] = 0;
            if (t >= total) continue;
            while (t >= first + q.n) {
                first += q.n;
                first_w += q.want;
                q = load_request(p, ++r);
            }
            const int at = q.ctx + t - first;
            const int blk = at / p.page_size;
            if (blk != page_blk || r != page_row) {  // tokens in a row mostly share a page
                page_blk = blk;
                page_row = r;
                page = -1;
                if (blk < q.held) page = p.table[(int64_t)r * p.max_blocks + blk];
                else if (blk < p.max_blocks && first_w + (blk - q.held) < count)
                    page = p.free_ring[ring_at(first_w + (blk - q.held))];
                if (page >= pages) page = -1;
            }
            if (page >= 0) slot[e] = page * p.page_size + at - blk * p.page_size;
            position[e] = at;
            if constexpr (kTree) position[e] = q.ctx + plan_node(p, t, first, t - first);
        }
        if constexpr (kTree) {
            if (t0 >= total && p.mask)
                for (int i = 0; i < p.mask_words; ++i) p.mask[(int64_t)t0 * p.mask_words + i] = 0u;
        }
        if (!kTree && vectors && t0 + kPer <= p.max_new) {
#pragma unroll
            for (int e = 0; e + 3 < kPer; e += 4) {
                *reinterpret_cast<int4 *>(p.slots + t0 + e) = make_int4(slot[e], slot[e + 1], slot[e + 2], slot[e + 3]);
                *reinterpret_cast<int4 *>(p.positions + t0 + e) =
                    make_int4(position[e], position[e + 1], position[e + 2], position[e + 3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (t0 + e < p.max_new) {
                    p.slots[t0 + e] = slot[e];
                    p.positions[t0 + e] = position[e];
                }
        }
    }
}

// ------------------------------------------------------------------ append
// A group of d / 8 threads moves one (token, head) row of K and of V, 16 bytes
// a thread and step, kRows rows at a time: the loads of the rows and of their
// slots are all under way before the first store needs them.  60,000 tokens of 8
// heads, bf16: 73 us, 6.72 TB/s, 99% of the copy rate (one row at a time: 78).
constexpr int kAppendThreads = 256, kAppendRows = 2;

template <int D, int kIn, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
    constexpr int kLanes = D / 8, kGroups = kAppendThreads / kLanes;
    griddep_wait();
    const float sk = kFp8 ? *p.scale_k : 1.f, sv = kFp8 ? *p.scale_v : 1.f;
    const int c = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int64_t rows = (int64_t)p.total * p.h_kv, step = (int64_t)gridDim.x * kGroups;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups + group; r0 < rows; r0 += step * kAppendRows) {
        uint4 a[kAppendRows], b[kAppendRows];
        int slot[kAppendRows], head[kAppendRows];
#pragma unroll
        for (int e = 0; e < kAppendRows; ++e) {
            const int64_t r = r0 + e * step;
            slot[e] = -1;
            if (r >= rows) continue;
            const int token = (int)r / p.h_kv;
            head[e] = (int)r - token * p.h_kv;
            slot[e] = p.slots[token];
            const int64_t src = head[e] * D + c * 8;
            a[e] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.k) + token * p.k_stride + src));
            b[e] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) + token * p.v_stride + src));
        }
#pragma unroll
        for (int e = 0; e < kAppendRows; ++e) {
            if (slot[e] < 0) continue;
            const int page = slot[e] / p.page_size, off = slot[e] - page * p.page_size;
            if (page >= p.num_pages) {
                report_bad_data(p.err, kTagCacheAppend, 1);
                continue;
            }
            const int64_t dst = (((int64_t)page * p.h_kv + head[e]) * p.page_size + off) * D + c * 8;
            if constexpr (!kFp8) {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.k_cache) + dst) = a[e];
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v_cache) + dst) = b[e];
            } else {
                auto codes = [](const uint4 &x, float s) {
                    const float2 f0 = unpack2<kIn == kElBf16>(x.x), f1 = unpack2<kIn == kElBf16>(x.y);
                    const float2 f2 = unpack2<kIn == kElBf16>(x.z), f3 = unpack2<kIn == kElBf16>(x.w);
                    return make_uint2(pack_e4m3x4(f0.x * s, f0.y * s, f1.x * s, f1.y * s),
                                      pack_e4m3x4(f2.x * s, f2.y * s, f3.x * s, f3.y * s));
                };
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.k_cache) + dst) = codes(a[e], sk);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.v_cache) + dst) = codes(b[e], sv);
            }
        }
    }
}

// ------------------------------------------------------------------ accept
// A CTA takes one request and up to 128 16-byte columns of its rows in the two
// caches; a thread owns a column and walks the path: the row of path[j] goes to
// row j.  path[j] >= j, so no row is overwritten before the walk has read it,
// and rows may be read ahead: kAcceptAhead of them, whose places the CTA looks
// up together (three dependent loads, which would be most of a row's time).
// 1000 requests that keep up to 12 of 64 nodes, 8 heads, bf16: 8.2 us, 4.9 TB/s
// (two rows ahead 9.6, eight 9.1, sixteen 12.1; 256 threads 8.5; one row after the
// other with its own look-ups 18.5).
constexpr int kAcceptAhead = 4;

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptParams p) {
    __shared__ int64_t s_from[kAcceptThreads], s_to[kAcceptThreads];  // row numbers of head 0, from < 0: no move
    griddep_wait();
    const int r = blockIdx.x;
    const int32_t *path = p.path + (int64_t)r * p.max_path;
    int node = (int)threadIdx.x < p.max_path ? path[threadIdx.x] : 0;  // with the lengths, not behind them
    const int fresh = max(p.fresh[r], 0);
    const int n = min(max(p.path_lens[r], 0), min(fresh, p.max_path));
    const int ctx = min(max(p.ctx[r], 0), INT32_MAX - fresh);
    if (blockIdx.y == 0 && threadIdx.x == 0) p.ctx_out[r] = ctx + n;
    const int chunks = p.row_bytes / 16, columns = 2 * p.h_kv * chunks;
    const int col = blockIdx.y * kAcceptThreads + threadIdx.x;
    const int which = col / (p.h_kv * chunks), head = col / chunks % p.h_kv, c = col % chunks;
    uint8_t *cache = static_cast<uint8_t *>(which ? p.v_cache : p.k_cache) + c * 16 +
                     (int64_t)head * p.page_size * p.row_bytes;
    auto place = [&](int pos) -> int64_t {
        const int blk = pos / p.page_size;
        const int page = blk < p.max_blocks ? p.table[(int64_t)r * p.max_blocks + blk] : -1;
        return page < 0 || page >= p.num_pages ? -1 : (int64_t)page * p.h_kv * p.page_size + pos % p.page_size;
    };
    for (int j0 = 0; j0 < n; j0 += kAcceptThreads) {
        const int j = j0 + threadIdx.x;
        if (j < n) {
            if (j0 > 0) node = path[j];
            int64_t from = -1, to = -1;
            if (node != j) {
                from = node > j && node < fresh ? place(ctx + node) : -1;
                to = place(ctx + j);
                if (from < 0 || to < 0) {
                    from = -1;
                    report_bad_data(p.err, kTagCacheAccept, 1);
                }
            }
            s_from[threadIdx.x] = from;
            s_to[threadIdx.x] = to;
        }
        __syncthreads();
        const int m = min(n - j0, kAcceptThreads);
        if (col < columns) {
            for (int k = 0; k < m; k += kAcceptAhead) {
                uint4 v[kAcceptAhead];
#pragma unroll
                for (int e = 0; e < kAcceptAhead; ++e)
                    if (k + e < m && s_from[k + e] >= 0) v[e] = *reinterpret_cast<const uint4 *>(cache + s_from[k + e] * p.row_bytes);
#pragma unroll
                for (int e = 0; e < kAcceptAhead; ++e)
                    if (k + e < m && s_from[k + e] >= 0) *reinterpret_cast<uint4 *>(cache + s_to[k + e] * p.row_bytes) = v[e];
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_cache_plan(const PlanParams &p, int sm_count, cudaStream_t stream) {
    const int64_t share = kPlanThreads * (p.parents ? 1 : kPlanTokens);
    const int64_t tokens = ((int64_t)p.max_new + share - 1) / share;
    const int64_t rows = ((int64_t)p.b + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    const int row_ctas = (int)(rows < 1 ? 1 : rows > sm_count ? sm_count : rows);
    const int token_ctas = (int)(tokens > 4 * sm_count ? 4 * sm_count : tokens);
    return launch_overlapped(p.parents ? plan_kernel<true> : plan_kernel<false>, dim3(row_ctas + token_ctas),
                             dim3(kPlanThreads), 0, stream, p, row_ctas);
}

cudaError_t launch_cache_append(const AppendParams &p, int dtype, int cache_dtype, cudaStream_t stream) {
    const int groups = kAppendThreads / (p.d / 8);
    // a CTA for each of its rows: a grid of 8 CTAs an SM that loops took 81 us for 60,000 tokens, this 74
    const int64_t grid = ((int64_t)p.total * p.h_kv + groups * kAppendRows - 1) / (groups * kAppendRows);
    auto run = [&](void (*kern)(const AppendParams)) {
        return launch_overlapped(kern, dim3((int)grid), dim3(kAppendThreads), 0, stream, p);
    };
    if (cache_dtype == kElE4m3) return run(dtype == kElBf16 ? append_kernel<128, kElBf16, true> : append_kernel<128, kElFp16, true>);
    return run(p.d == 64 ? append_kernel<64, kElBf16, false> : append_kernel<128, kElBf16, false>);
}

cudaError_t launch_cache_accept(const AcceptParams &p, cudaStream_t stream) {
    const int columns = 2 * p.h_kv * (p.row_bytes / 16);
    return launch_overlapped(accept_kernel, dim3(p.b, (columns + kAcceptThreads - 1) / kAcceptThreads), dim3(kAcceptThreads),
                             0, stream, p);
}

}  // namespace sdpa
