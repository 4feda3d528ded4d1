// Eviction from a paged cache by accumulated attention weight (kv_evict / kv_evict_fp8).
//
// For a sequence of L > keep cells and each KV head: the first f and the last r cells stay; of
// the middle cells [f, L - r) the n = keep - f - r of largest weight stay (ties: the lowest
// cell). A cell is moved only if it has to be: kept middle cells at or beyond f + n ("surplus",
// ascending) go into the freed cells below f + n ("holes", ascending, as many), and the last r
// cells go to [keep - r, keep) in order. So a cache that outgrew its size by a few cells moves
// a few cells and the last r, not all it keeps.
//
// One cluster of CTAs per (sequence, KV head), the warps of the cluster holding consecutive
// runs of cells:
//   1. weights -> order-preserving 32-bit keys (in shared memory when they fit)
//   2. the n-th largest key by four 8-bit histogram rounds, the CTAs' histograms added up
//      through distributed shared memory
//   3. tallies per warp, their prefix over the cluster: every warp knows how many ties, holes
//      and surplus cells lie before its run
//   4. each warp lists its holes and surplus cells, in order (workspace)
//   5. surplus -> holes: sources and destinations are disjoint, all moves at once
//   6. the last r cells, a round of rows at a time: read, cluster barrier, write. A source lies
//      above its destination, so a round's writes never touch a later round's sources.
// Bound by HBM on the moved rows and the weights, by the rounds' latency when few cells move.

constexpr int kEvWarps = 16;
constexpr int kEvThreads = kEvWarps * 32;
constexpr int kEvMaxCluster = 8;                // portable cluster size
constexpr int kEvMaxKeys = 48 * 1024;           // keys one CTA holds in shared memory at most
constexpr int kEvUnroll = 4;                    // rows in flight per half-warp

struct EvictParams {
    uint8_t *k_cache, *v_cache;  // fp8: k_cache holds the blocks
    float *weights;              // [num_pages][Hkv][16]
    const int *block_table, *seq_lens;
    int *new_lens, *kept;        // [B], [B][Hkv][keep]
    int2 *lists;                 // [B * Hkv][2][keep]: holes, surplus, as (cell, page)
    int Hkv, keep, first, last, max_pages, num_pages, max_seq_len;
    int key_cap;                 // keys a CTA's shared memory holds
};

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ uint32_t cluster_ld(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Order-preserving key of a weight: larger weight, larger key; -0 equals +0; NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One row (a cell's K, V and weight) on its way from one cell to another, held by the 16 lanes
// of a half-warp. bf16: lanes 0-7 a 16-byte piece of K each, 8-15 of V. fp8 blocks: every lane
// 4 bytes of the V column (one per row of V^T), lanes 0-3 a piece of the K row, 4 and 5 the
// scales. The weight rides with lane 6.
template <bool KV8>
struct EvRow {
    uint4 kv;
    uint32_t col;
    float w;
};

template <bool KV8>
__device__ __forceinline__ void ev_load(const EvictParams &p, EvRow<KV8> &row, int page, int slot, int g, int hl) {
    const size_t tile = static_cast<size_t>(page) * p.Hkv + g;
    if constexpr (KV8) {
        const uint8_t *blk = p.k_cache + tile * kBlk8Bytes;
        const uint8_t *v = blk + kBlk8V + 4 * hl * kPage + slot;
        row.col = v[0] | (v[kPage] << 8) | (v[2 * kPage] << 16) | (static_cast<uint32_t>(v[3 * kPage]) << 24);
        if (hl < 4) row.kv = *reinterpret_cast<const uint4 *>(blk + slot * kD + 16 * hl);
        if (hl == 4 || hl == 5) row.w = reinterpret_cast<const float *>(blk + kBlk8S)[(hl - 4) * kPage + slot];
    } else {
        const uint8_t *src = (hl < 8 ? p.k_cache : p.v_cache) + (tile * kPage + slot) * (kD * 2) + 16 * (hl & 7);
        row.kv = *reinterpret_cast<const uint4 *>(src);
    }
    if (hl == 6) row.w = p.weights[tile * kPage + slot];
}

template <bool KV8>
__device__ __forceinline__ void ev_store(const EvictParams &p, const EvRow<KV8> &row, int page, int slot, int g, int hl) {
    const size_t tile = static_cast<size_t>(page) * p.Hkv + g;
    if constexpr (KV8) {
        uint8_t *blk = p.k_cache + tile * kBlk8Bytes;
        uint8_t *v = blk + kBlk8V + 4 * hl * kPage + slot;
        v[0] = static_cast<uint8_t>(row.col);
        v[kPage] = static_cast<uint8_t>(row.col >> 8);
        v[2 * kPage] = static_cast<uint8_t>(row.col >> 16);
        v[3 * kPage] = static_cast<uint8_t>(row.col >> 24);
        if (hl < 4) *reinterpret_cast<uint4 *>(blk + slot * kD + 16 * hl) = row.kv;
        if (hl == 4 || hl == 5) reinterpret_cast<float *>(blk + kBlk8S)[(hl - 4) * kPage + slot] = row.w;
    } else {
        uint8_t *dst = (hl < 8 ? p.k_cache : p.v_cache) + (tile * kPage + slot) * (kD * 2) + 16 * (hl & 7);
        *reinterpret_cast<uint4 *>(dst) = row.kv;
    }
    if (hl == 6) p.weights[tile * kPage + slot] = row.w;
}

template <bool KV8>
__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[4][256];
    __shared__ int4 s_tally[kEvWarps];                   // gt_lo, eq_lo, gt_hi, eq_hi of each warp
    __shared__ int4 s_all[kEvWarps * kEvMaxCluster];     // the cluster's tallies, then the prefixes
    __shared__ uint32_t s_wsum[8];
    __shared__ uint32_t s_digit, s_want;
    __shared__ int s_moves;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = gridDim.x, rank = blockIdx.x;          // the cluster spans the grid's x
    const int g = blockIdx.y, b = blockIdx.z;
    for (int i = tid; i < 4 * 256; i += kEvThreads) (&s_hist[0][0])[i] = 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const size_t pair = static_cast<size_t>(b) * p.Hkv + g;
    int *const kept = p.kept + pair * p.keep;
    int L = __ldg(p.seq_lens + b);
    if (L < 0 || L > p.max_seq_len || L > p.max_pages * kPage) {
        if (tid == 0 && rank == 0 && g == 0) flag_status(DA_STATUS_BAD_SEQ_LEN);
        L = 0;
    }
    if (tid == 0 && rank == 0 && g == 0) p.new_lens[b] = min(L, p.keep);
    if (L <= p.keep) {  // (every CTA of the cluster leaves here or none)
        for (int i = rank * kEvThreads + tid; i < p.keep; i += C * kEvThreads) kept[i] = i < L ? i : -1;
        return;
    }
    const int f = p.first, r = p.last, n = p.keep - f - r;
    const int m0 = f, m1 = L - r, low = f + n;           // the middle cells, and where they may stay
    const int *const bt = p.block_table + static_cast<size_t>(b) * p.max_pages;

    // ---- 1. this warp's run of cells [c0, c1) (32 at a time), the CTA's first cell
    const int chunks = (L + 31) / 32, cpw = (chunks + C * kEvWarps - 1) / (C * kEvWarps);
    const int cta0 = rank * kEvWarps * cpw * 32;
    const int c0 = cta0 + warp * cpw * 32, c1 = min(c0 + cpw * 32, L);
    const bool resident = kEvWarps * cpw * 32 <= p.key_cap;
    auto page_of = [&](int cell) {
        const int page = __ldg(bt + cell / kPage);
        return page >= 0 && page < p.num_pages ? page : -1;
    };
    auto load_key = [&](int cell) -> uint32_t {
        const int page = page_of(cell);
        if (page < 0) {
            flag_status(DA_STATUS_BAD_PAGE);
            return 0u;
        }
        return weight_key(p.weights[(static_cast<size_t>(page) * p.Hkv + g) * kPage + cell % kPage]);
    };
    auto key_of = [&](int cell) { return resident ? s_key[cell - cta0] : load_key(cell); };
    __syncthreads();  // (the histograms are zero)
#pragma unroll 4
    for (int c = c0 + lane; c < c1; c += 32) {
        const uint32_t key = load_key(c);
        if (resident) s_key[c - cta0] = key;
        if (c >= m0 && c < m1) atomicAdd(&s_hist[0][key >> 24], 1u);
    }

    // ---- 2. the n-th largest key of the middle: thr, and how many cells of exactly that key stay
    uint32_t thr = 0xffffffffu, ties = 0;
    if (n > 0) {
        uint32_t prefix = 0, want = n;
#pragma unroll 1
        for (int round = 0; round < 4; ++round) {
            const int sh = 24 - 8 * round;
            if (round > 0) {
                for (int c = c0 + lane; c < c1; c += 32) {
                    const uint32_t key = key_of(c);
                    if (c >= m0 && c < m1 && (key >> (sh + 8)) == prefix) atomicAdd(&s_hist[round][(key >> sh) & 255u], 1u);
                }
            }
            cluster_sync_all();
            uint32_t cnt = 0, incl = 0;
            if (tid < 256) {  // bin 255 - tid, summed over the cluster, scanned from the top
                const uint32_t a = smem_addr(&s_hist[round][255 - tid]);
                for (int k = 0; k < C; ++k) cnt += cluster_ld(cluster_map(a, k));
                incl = cnt;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += y;
                }
                if (lane == 31) s_wsum[warp] = incl;
            }
            __syncthreads();
            if (tid < 256) {
                for (int w = 0; w < warp; ++w) incl += s_wsum[w];
                if (incl >= want && incl - cnt < want) {  // exactly one bin
                    s_digit = 255 - tid;
                    s_want = want - (incl - cnt);
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | s_digit;
            want = s_want;
        }
        thr = prefix;
        ties = want;
    }

    // ---- 3. tallies: keys above and at the threshold, below and beyond `low`
    int gt_lo = 0, eq_lo = 0, gt_hi = 0, eq_hi = 0;
    for (int c = c0; c < c1; c += 32) {
        const int cell = c + lane;
        const bool mid = cell < c1 && cell >= m0 && cell < m1;
        const uint32_t key = mid ? key_of(cell) : 0u;
        const bool lo = cell < low;
        gt_lo += __popc(__ballot_sync(0xffffffffu, mid && lo && key > thr));
        eq_lo += __popc(__ballot_sync(0xffffffffu, mid && lo && key == thr));
        gt_hi += __popc(__ballot_sync(0xffffffffu, mid && !lo && key > thr));
        eq_hi += __popc(__ballot_sync(0xffffffffu, mid && !lo && key == thr));
    }
    if (lane == 0) s_tally[warp] = make_int4(gt_lo, eq_lo, gt_hi, eq_hi);
    cluster_sync_all();
    if (tid < C * kEvWarps) {
        const uint32_t a = cluster_map(smem_addr(&s_tally[tid % kEvWarps]), tid / kEvWarps);
        s_all[tid] = make_int4(cluster_ld(a), cluster_ld(a + 4), cluster_ld(a + 8), cluster_ld(a + 12));
    }
    __syncthreads();
    if (warp == 0) {  // ties, holes and surplus cells before each warp's run
        int eq_run = 0, hole_run = 0, more_run = 0;
        for (int w0 = 0; w0 < C * kEvWarps; w0 += 32) {
            const int w = w0 + lane;
            const int4 t = w < C * kEvWarps ? s_all[w] : make_int4(0, 0, 0, 0);
            auto scan = [&](int v) {
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, v, off);
                    if (lane >= off) v += y;
                }
                return v;
            };
            const int eq = t.y + t.w, eq_in = scan(eq), eq_before = eq_run + eq_in - eq;
            const int left = max(0, static_cast<int>(ties) - eq_before);
            const int eq_kept_lo = min(left, t.y), eq_kept_hi = min(left - eq_kept_lo, t.w);
            const int a = max(w * cpw * 32, m0), e = min((w + 1) * cpw * 32, low);
            const int holes = max(0, e - a) - t.x - eq_kept_lo, more = t.z + eq_kept_hi;
            const int holes_in = scan(holes), more_in = scan(more);
            if (w < C * kEvWarps) s_all[w] = make_int4(eq_before, hole_run + holes_in - holes, more_run + more_in - more, 0);
            eq_run += __shfl_sync(0xffffffffu, eq_in, 31);
            hole_run += __shfl_sync(0xffffffffu, holes_in, 31);
            more_run += __shfl_sync(0xffffffffu, more_in, 31);
        }
        if (lane == 0) s_moves = hole_run;
    }
    __syncthreads();
    const int moves = s_moves;

    // ---- 4. the holes and the surplus cells, in order
    int2 *const holes = p.lists + pair * 2 * p.keep, *const surplus = holes + p.keep;
    {
        const int4 pre = s_all[rank * kEvWarps + warp];
        int eq_at = pre.x, hole_at = pre.y, more_at = pre.z;
        const uint32_t below = (1u << lane) - 1u;
        for (int c = c0; c < c1; c += 32) {
            const int cell = c + lane;
            const bool mid = cell < c1 && cell >= m0 && cell < m1;
            const uint32_t key = mid ? key_of(cell) : 0u;
            const bool eq = mid && key == thr;
            const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
            const bool stay = mid && (key > thr || (eq && eq_at + __popc(eqs & below) < static_cast<int>(ties)));
            const bool hole = mid && !stay && cell < low, more = stay && cell >= low;
            const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, more);
            if (hole) holes[hole_at + __popc(hs & below)] = make_int2(cell, page_of(cell));
            if (more) surplus[more_at + __popc(ms & below)] = make_int2(cell, page_of(cell));
            if (cell < m0 || (stay && cell < low)) kept[cell] = cell;
            eq_at += __popc(eqs);
            hole_at += __popc(hs);
            more_at += __popc(ms);
        }
    }
    cluster_sync_all();

    // ---- 5. surplus cells into the holes
    const int hl = lane & 15;
    const int halves = 2 * kEvWarps * C, half = 2 * (rank * kEvWarps + warp) + (lane >> 4);
    for (int j0 = half; j0 < moves; j0 += halves * kEvUnroll) {
        EvRow<KV8> row[kEvUnroll];
        int2 to[kEvUnroll], from[kEvUnroll];
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
            const int j = j0 + u * halves;
            to[u] = from[u] = make_int2(0, -1);
            if (j < moves) {
                to[u] = __ldcg(holes + j);
                from[u] = __ldcg(surplus + j);
            }
        }
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u)
            if (from[u].y >= 0) ev_load(p, row[u], from[u].y, from[u].x % kPage, g, hl);
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
            if (j0 + u * halves < moves && hl == 7) kept[to[u].x] = from[u].x;
            if (from[u].y >= 0 && to[u].y >= 0) ev_store(p, row[u], to[u].y, to[u].x % kPage, g, hl);
        }
    }

    // ---- 6. the last r cells, a round of rows at a time. The first barrier also lets step 5 finish
    // reading the surplus cells that the rows are written over.
    const int shift = L - p.keep;
    const bool overlap = shift < r;  // (else no later round's sources lie where this one writes)
    const int per_round = halves * kEvUnroll;
    for (int i0 = 0; i0 < r; i0 += per_round) {
        EvRow<KV8> row[kEvUnroll];
        int from[kEvUnroll], to[kEvUnroll];
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
            const int i = i0 + half + u * halves;
            from[u] = to[u] = -1;
            if (i < r) {
                const int dst = p.keep - r + i;
                from[u] = page_of(dst + shift);
                to[u] = page_of(dst);
                if (hl == 7) kept[dst] = dst + shift;
                if (from[u] >= 0) ev_load(p, row[u], from[u], (dst + shift) % kPage, g, hl);
            }
        }
        if (i0 == 0 || overlap) cluster_sync_all();
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
            const int i = i0 + half + u * halves;
            if (i < r && from[u] >= 0 && to[u] >= 0) ev_store(p, row[u], to[u], (p.keep - r + i) % kPage, g, hl);
        }
    }
}
