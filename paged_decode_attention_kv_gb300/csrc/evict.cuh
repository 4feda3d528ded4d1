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
//   2. the n-th largest key by up to three histogram rounds (11, 11 and 10 bits; the first digit
//      then holds two bits of the mantissa, so that weights of a few octaves do not all count
//      in a few bins); the CTAs of a cluster add theirs up in global memory (L2: every CTA reading
//      all 2048 bins of all others through distributed shared memory took 5 us a round)
//   3. tallies per warp, their prefix over the cluster: every warp knows how many ties, holes
//      and surplus cells lie before its run
//   4. each warp lists its holes and surplus cells, in order (workspace): a lane has the ballots of
//      one 32-cell chunk, so the lists cost a few instructions per cell listed, not per cell
//   5. surplus -> holes: sources and destinations are disjoint, all moves at once. fp8 blocks hold V
//      transposed, a token's V in 64 places: there a warp takes a destination tile, puts the
//      sources' bytes into its rows in registers and writes the tile's rows once (a byte store
//      per value took twice as long)
//   6. the last r cells, a round of rows at a time: read, cluster barrier, write. A source lies
//      above its destination, so a round's writes never touch a later round's sources.
// Bound by HBM on the moved rows and the weights, by the rounds' latency when few cells move.

// CTAs have 16 warps (two on an SM), or 32 and work in clusters for a few long sequences.
constexpr int kEvMaxWarps = 32;
constexpr int kEvMaxCluster = 16;               // (over 8: where the device takes it)
constexpr int kEvMaxKeys = 48 * 1024;           // keys one CTA holds in shared memory at most
constexpr int kEvUnroll = 4;                    // rows in flight per half-warp
constexpr int kEvTileUnroll = 4;                // fp8: sources in flight per warp
constexpr int kEvLoad = 16;                     // weights in flight per lane
constexpr int kEvBins = 2048;
constexpr int kEvMaxBins = kEvBins / 512;       // per thread
constexpr int kEvClusterPairs = kMaxSms / 2;    // clusters have two CTAs or more, at most one per SM
constexpr size_t kEvHistBytes = static_cast<size_t>(kEvClusterPairs) * 3 * kEvBins * 4;  // ahead of the workspace

struct EvictParams {
    uint8_t *k_cache, *v_cache;  // fp8: k_cache holds the blocks
    float *weights;              // [num_pages][Hkv][16]
    const int *block_table, *seq_lens;
    int *new_lens, *kept;        // [B], [B][Hkv][keep]
    int *lists;                  // [B * Hkv][evict_list_ints(keep)]: holes, surplus cells, and for each
                                 // tile the number of holes before it
    uint32_t *hist;              // clusters: [B * Hkv][3][kEvBins], zero at rest
    int Hkv, keep, first, last, max_pages, num_pages, max_seq_len;
    int key_cap;                 // keys a CTA's shared memory holds
};

__host__ __device__ constexpr size_t evict_list_ints(int keep) {
    return 2 * static_cast<size_t>(keep) + (keep + kPage - 1) / kPage;
}

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
__global__ void __launch_bounds__(kEvMaxWarps * 32) kv_evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[2][kEvBins];
    __shared__ int4 s_tally[kEvMaxWarps];                  // gt_lo, eq_lo, gt_hi, eq_hi of each warp
    __shared__ int4 s_all[kEvMaxWarps * kEvMaxCluster];    // the cluster's tallies, then the prefixes
    __shared__ uint32_t s_wsum[kEvMaxWarps];
    __shared__ uint32_t s_digit, s_want, s_cnt;
    __shared__ int s_moves;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nt = blockDim.x, nwarps = nt >> 5;
    const int C = gridDim.x, rank = blockIdx.x;            // the cluster spans the grid's x
    const int g = blockIdx.y, b = blockIdx.z;
    auto sync_cluster = [&]() {
        if (C > 1) cluster_sync_all();
        else __syncthreads();
    };
    for (int i = tid; i < 2 * kEvBins; i += nt) (&s_hist[0][0])[i] = 0u;
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
        for (int i = rank * nt + tid; i < p.keep; i += C * nt) kept[i] = i < L ? i : -1;
        return;
    }
    const int f = p.first, r = p.last, n = p.keep - f - r;
    const int m0 = f, m1 = L - r, low = f + n;             // the middle cells, and where they may stay
    const int *const bt = p.block_table + static_cast<size_t>(b) * p.max_pages;

    // ---- 1. this warp's run of cells [c0, c1) (32 at a time), the CTA's first cell
    const int chunks = (L + 31) / 32, cpw = (chunks + C * nwarps - 1) / (C * nwarps);
    const int cta0 = rank * nwarps * cpw * 32;
    const int c0 = cta0 + warp * cpw * 32, c1 = min(c0 + cpw * 32, L);
    const bool resident = nwarps * cpw * 32 <= p.key_cap;
    auto page_of = [&](int cell) {
        const int page = __ldg(bt + cell / kPage);
        return page >= 0 && page < p.num_pages ? page : -1;
    };
    auto key_at = [&](int cell, int page) {
        return page < 0 ? 0u : weight_key(p.weights[(static_cast<size_t>(page) * p.Hkv + g) * kPage + cell % kPage]);
    };
    auto key_of = [&](int cell) { return resident ? s_key[cell - cta0] : key_at(cell, page_of(cell)); };
    uint32_t *const ghist = p.hist + pair * (3 * kEvBins);
    int rounds = 0;                                        // histogram rounds made
    __syncthreads();  // (the histograms are zero)
    for (int cb = c0; cb < c1; cb += 512) {                // 16 chunks: their 32 pages at once, one per lane
        int pages = -1;
        if (cb + 16 * lane < c1) {
            pages = page_of(cb + 16 * lane);
            if (pages < 0) flag_status(DA_STATUS_BAD_PAGE);
        }
#pragma unroll
        for (int u = 0; u < 16; u += kEvLoad) {
            if (cb + 32 * u >= c1) break;
            uint32_t key[kEvLoad];
#pragma unroll
            for (int k = 0; k < kEvLoad; ++k) {
                const int cell = cb + 32 * (u + k) + lane;
                const int page = __shfl_sync(0xffffffffu, pages, 2 * (u + k) + (lane >> 4));
                key[k] = cell < c1 ? key_at(cell, page) : 0u;
            }
#pragma unroll
            for (int k = 0; k < kEvLoad; ++k) {
                const int cell = cb + 32 * (u + k) + lane;
                if (cell < c1) {
                    if (resident) s_key[cell - cta0] = key[k];
                    if (cell >= m0 && cell < m1) atomicAdd(&s_hist[0][key[k] >> 21], 1u);
                }
            }
        }
    }

    // ---- 2. the n-th largest key of the middle: cells above thr stay, and `ties` of those at it
    uint32_t thr = 0xffffffffu, ties = 0;
    if (n > 0) {
        uint32_t prefix = 0, want = n;
#pragma unroll 1
        for (int round = 0; round < 3; ++round) {
            const int sh = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round < 2 ? 11 : 10;
            uint32_t *const hist = s_hist[round & 1];
            if (round > 0) {
                for (int c = c0 + lane; c < c1; c += 32) {
                    const uint32_t key = key_of(c);
                    if (c >= m0 && c < m1 && (key >> (sh + bits)) == prefix) atomicAdd(&hist[(key >> sh) & ((1u << bits) - 1u)], 1u);
                }
            }
            const int per = kEvBins / nt;                  // consecutive bins per thread, from the top
            uint32_t cnt[kEvMaxBins], sum = 0;
            __syncthreads();
            rounds = round + 1;
            if (C > 1) {
                uint32_t *const all = ghist + round * kEvBins;
                for (int i = tid; i < kEvBins; i += nt)
                    if (hist[i] != 0u) atomicAdd(all + i, hist[i]);
                sync_cluster();
#pragma unroll
                for (int k = 0; k < kEvMaxBins; ++k) cnt[k] = k < per ? __ldcg(all + kEvBins - 1 - (tid * per + k)) : 0u;
            } else {
#pragma unroll
                for (int k = 0; k < kEvMaxBins; ++k) cnt[k] = k < per ? hist[kEvBins - 1 - (tid * per + k)] : 0u;
            }
#pragma unroll
            for (int k = 0; k < kEvMaxBins; ++k) sum += cnt[k];
            uint32_t incl = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            if (lane == 31) s_wsum[warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += s_wsum[w];
            if (incl >= want && incl - sum < want) {       // exactly one thread: the bin is among its own
                uint32_t above = incl - sum;
                bool found = false;
#pragma unroll
                for (int k = 0; k < kEvMaxBins; ++k) {
                    if (!found && above + cnt[k] >= want) {
                        found = true;
                        s_digit = kEvBins - 1 - (tid * per + k);
                        s_want = want - above;
                        s_cnt = cnt[k];
                    }
                    above += cnt[k];
                }
            }
            __syncthreads();
            prefix = (prefix << bits) | s_digit;
            want = s_want;
            if (sh > 0 && s_cnt == want && prefix > 0) {   // the whole bin stays: no need to look into it
                thr = (prefix << sh) - 1u;
                break;
            }
            if (sh == 0) {
                thr = prefix;
                ties = want;
            } else if (round == 1) {                       // the third round counts where the first did
                for (int i = tid; i < kEvBins; i += nt) s_hist[0][i] = 0u;
                __syncthreads();
            }
        }
    }

    // ---- 3. tallies: keys above and at the threshold, below and beyond `low`. Lane l holds the masks
    // of chunk l of the run's block of 32 chunks (a run of more blocks works them out again in 4).
    auto bits_below = [](int x) { return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u; };
    auto block_masks = [&](int cb, uint32_t &gt, uint32_t &eq) {
        gt = eq = 0u;
        const int cnt = min(32, (c1 - cb + 31) / 32);
        for (int i = 0; i < cnt; ++i) {
            const int cell = cb + 32 * i + lane;
            const bool mid = cell < c1 && cell >= m0 && cell < m1;
            const uint32_t key = mid ? key_of(cell) : 0u;
            const uint32_t g_ = __ballot_sync(0xffffffffu, mid && key > thr), e_ = __ballot_sync(0xffffffffu, mid && key == thr);
            if (lane == i) {
                gt = g_;
                eq = e_;
            }
        }
    };
    uint32_t gt = 0u, eq = 0u;
    {
        int4 t = make_int4(0, 0, 0, 0);
        for (int cb = c0; cb < c1; cb += 1024) {
            block_masks(cb, gt, eq);
            const uint32_t lo = bits_below(low - (cb + 32 * lane));
            t.x += __popc(gt & lo);
            t.y += __popc(eq & lo);
            t.z += __popc(gt & ~lo);
            t.w += __popc(eq & ~lo);
        }
        t.x = __reduce_add_sync(0xffffffffu, t.x);
        t.y = __reduce_add_sync(0xffffffffu, t.y);
        t.z = __reduce_add_sync(0xffffffffu, t.z);
        t.w = __reduce_add_sync(0xffffffffu, t.w);
        if (lane == 0) s_tally[warp] = t;
    }
    sync_cluster();
    if (C > 1)  // every CTA has read the sums: zero again for the next call
        for (int i = rank * nt + tid; i < rounds * kEvBins; i += C * nt) ghist[i] = 0u;
    if (tid < C * nwarps) {
        const uint32_t a = cluster_map(smem_addr(&s_tally[tid % nwarps]), tid / nwarps);
        s_all[tid] = make_int4(cluster_ld(a), cluster_ld(a + 4), cluster_ld(a + 8), cluster_ld(a + 12));
    }
    __syncthreads();
    if (warp == 0) {  // ties, holes and surplus cells before each warp's run: consecutive runs per lane
        constexpr int kPer = 8;
        auto scan = [&](int v) {                           // exclusive prefix over the lanes
            int x = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            return x - v;
        };
        int eq_run = 0, hole_run = 0, more_run = 0;
        for (int first = 0; first < C * nwarps; first += 32 * kPer) {
            const int w0 = first + lane * kPer;
            int4 t[kPer];
            int eq_sum = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                t[k] = w0 + k < C * nwarps ? s_all[w0 + k] : make_int4(0, 0, 0, 0);
                eq_sum += t[k].y + t[k].w;
            }
            int eq_at = eq_run + scan(eq_sum), hole_sum = 0, more_sum = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {               // t becomes (ties before, holes, surplus)
                const int left = max(0, static_cast<int>(ties) - eq_at);
                const int eq_lo = min(left, t[k].y), eq_hi = min(left - eq_lo, t[k].w);
                const int a = max((w0 + k) * cpw * 32, m0), e = min((w0 + k + 1) * cpw * 32, low);
                const int holes = w0 + k < C * nwarps ? max(0, e - a) - t[k].x - eq_lo : 0, more = t[k].z + eq_hi;
                const int eq = t[k].y + t[k].w;
                t[k] = make_int4(eq_at, holes, more, 0);
                eq_at += eq;
                hole_sum += holes;
                more_sum += more;
            }
            int hole_at = hole_run + scan(hole_sum), more_at = more_run + scan(more_sum);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                if (w0 + k < C * nwarps) s_all[w0 + k] = make_int4(t[k].x, hole_at, more_at, 0);
                hole_at += t[k].y;
                more_at += t[k].z;
            }
            eq_run = __shfl_sync(0xffffffffu, eq_at, 31);
            hole_run = __shfl_sync(0xffffffffu, hole_at, 31);
            more_run = __shfl_sync(0xffffffffu, more_at, 31);
        }
        if (lane == 0) s_moves = hole_run;
    }
    __syncthreads();
    const int moves = s_moves;

    // ---- 4. the holes and the surplus cells, in order
    int *const holes = p.lists + pair * evict_list_ints(p.keep), *const surplus = holes + p.keep;
    int *const before = surplus + p.keep;                  // holes before each tile
    auto scan_lanes = [&](int v) {                         // exclusive prefix over the lanes; total in lane 31's v + prefix
        int x = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        return x - v;
    };
    {
        const int4 pre = s_all[rank * nwarps + warp];
        int eq_at = pre.x, hole_at = pre.y, more_at = pre.z;
        for (int cb = c0; cb < c1; cb += 1024) {
            if (c1 - c0 > 1024) block_masks(cb, gt, eq);
            const int base = cb + 32 * lane;               // this lane's chunk
            const uint32_t lo = bits_below(low - base);
            const uint32_t mid = base < c1 ? bits_below(min(m1, c1) - base) & ~bits_below(m0 - base) : 0u;
            const int eqs = __popc(eq), eq_first = eq_at + scan_lanes(eqs);
            // of the ties, the lowest cells stay
            uint32_t eq_stay = eq;
            for (int drop = eqs - max(0, min(eqs, static_cast<int>(ties) - eq_first)); drop > 0; --drop)
                eq_stay &= ~(0x80000000u >> __clz(eq_stay));
            const uint32_t stay = gt | eq_stay;
            uint32_t hole = mid & ~stay & lo, more = stay & ~lo;
            const int nh = __popc(hole), nm = __popc(more);
            int h = hole_at + scan_lanes(nh), m = more_at + scan_lanes(nm);
            eq_at = __shfl_sync(0xffffffffu, eq_first + eqs, 31);
            hole_at = __shfl_sync(0xffffffffu, h + nh, 31);
            more_at = __shfl_sync(0xffffffffu, m + nm, 31);
            if (base < c1) {
                if (base < p.keep) before[base / kPage] = h;
                if (base + kPage < p.keep) before[base / kPage + 1] = h + __popc(hole & 0xffffu);
            }
            for (; hole; hole &= hole - 1) holes[h++] = base + __ffs(hole) - 1;
            for (; more; more &= more - 1) surplus[m++] = base + __ffs(more) - 1;
            const uint32_t same = base < c1 ? (stay & lo) | bits_below(m0 - base) : 0u;
            for (int i = 0; i < 32 && cb + 32 * i < min(c1, low); ++i)
                if (__shfl_sync(0xffffffffu, same, i) >> lane & 1u) kept[cb + 32 * i + lane] = cb + 32 * i + lane;
        }
    }
    sync_cluster();

    // ---- 5. surplus cells into the holes
    const int hl = lane & 15;
    const int halves = 2 * nwarps * C, half = 2 * (rank * nwarps + warp) + (lane >> 4);
    if constexpr (KV8) {
        const int tiles = (low + kPage - 1) / kPage;
        for (int t = rank * nwarps + warp; t < tiles; t += C * nwarps) {
            const int h0 = __ldcg(before + t), cnt = (t + 1 < tiles ? __ldcg(before + t + 1) : moves) - h0;
            if (cnt == 0) continue;
            // lane i: slot of the tile's i-th hole, slot and tile (-1: bad page) its token comes from
            int slots = 0, src_tile = -1;
            if (lane < cnt) {
                const int to = __ldcg(holes + h0 + lane), from = __ldcg(surplus + h0 + lane);
                kept[to] = from;
                const int page = page_of(from);
                src_tile = page < 0 ? -1 : page * p.Hkv + g;
                slots = to % kPage | (from % kPage) << 8;
            }
            const int dst = page_of(t * kPage);
            if (dst < 0) continue;
            const size_t dst_tile = static_cast<size_t>(dst) * p.Hkv + g;
            uint8_t *blk = p.k_cache + dst_tile * kBlk8Bytes;
            uint4 *vrow = reinterpret_cast<uint4 *>(blk + kBlk8V);
            uint4 v[2] = {vrow[lane], vrow[lane + 32]};    // rows d = lane, lane + 32 of V^T
            for (int i0 = 0; i0 < cnt; i0 += kEvTileUnroll) {
                uint4 krow[kEvTileUnroll];
                uint32_t src[kEvTileUnroll][2];            // the words of rows lane, lane + 32 that hold the byte
                float x[kEvTileUnroll];
                int tile[kEvTileUnroll], sl[kEvTileUnroll];
#pragma unroll
                for (int u = 0; u < kEvTileUnroll; ++u) {
                    tile[u] = __shfl_sync(0xffffffffu, src_tile, min(i0 + u, cnt - 1));
                    sl[u] = __shfl_sync(0xffffffffu, slots, min(i0 + u, cnt - 1));
                    if (i0 + u >= cnt) tile[u] = -1;
                    if (tile[u] >= 0) {
                        const int ss = sl[u] >> 8;
                        const uint8_t *from_blk = p.k_cache + static_cast<size_t>(tile[u]) * kBlk8Bytes;
                        const uint32_t *vs = reinterpret_cast<const uint32_t *>(from_blk + kBlk8V) + (ss >> 2) + 4 * lane;
                        src[u][0] = vs[0];
                        src[u][1] = vs[128];
                        if (lane < 4) krow[u] = *reinterpret_cast<const uint4 *>(from_blk + ss * kD + 16 * lane);
                        if (lane == 4 || lane == 5) x[u] = reinterpret_cast<const float *>(from_blk + kBlk8S)[(lane - 4) * kPage + ss];
                        if (lane == 6) x[u] = p.weights[static_cast<size_t>(tile[u]) * kPage + ss];
                    }
                }
#pragma unroll
                for (int u = 0; u < kEvTileUnroll; ++u) {
                    if (tile[u] < 0) continue;
                    const int ss = sl[u] >> 8, sd = sl[u] & 255;
                    // byte ss % 4 of the source's word into byte sd % 4 of word sd / 4 of the row
                    const int at = 4 * (sd & 3);
                    const uint32_t pick = (0x3210u & ~(15u << at)) | (4u + (ss & 3)) << at;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (sd < 4) v[k].x = __byte_perm(v[k].x, src[u][k], pick);
                        else if (sd < 8) v[k].y = __byte_perm(v[k].y, src[u][k], pick);
                        else if (sd < 12) v[k].z = __byte_perm(v[k].z, src[u][k], pick);
                        else v[k].w = __byte_perm(v[k].w, src[u][k], pick);
                    }
                    if (lane < 4) *reinterpret_cast<uint4 *>(blk + sd * kD + 16 * lane) = krow[u];
                    if (lane == 4 || lane == 5) reinterpret_cast<float *>(blk + kBlk8S)[(lane - 4) * kPage + sd] = x[u];
                    if (lane == 6) p.weights[dst_tile * kPage + sd] = x[u];
                }
            }
            vrow[lane] = v[0];
            vrow[lane + 32] = v[1];
        }
    } else {
        for (int j0 = half; j0 < moves; j0 += halves * kEvUnroll) {
            EvRow<KV8> row[kEvUnroll];
            int to[kEvUnroll], from[kEvUnroll], pt[kEvUnroll], pf[kEvUnroll];
#pragma unroll
            for (int u = 0; u < kEvUnroll; ++u) {
                const int j = j0 + u * halves;
                to[u] = j < moves ? __ldcg(holes + j) : -1;
                from[u] = j < moves ? __ldcg(surplus + j) : -1;
            }
#pragma unroll
            for (int u = 0; u < kEvUnroll; ++u) {
                pt[u] = to[u] >= 0 ? page_of(to[u]) : -1;
                pf[u] = from[u] >= 0 ? page_of(from[u]) : -1;
            }
#pragma unroll
            for (int u = 0; u < kEvUnroll; ++u)
                if (pf[u] >= 0) ev_load(p, row[u], pf[u], from[u] % kPage, g, hl);
#pragma unroll
            for (int u = 0; u < kEvUnroll; ++u) {
                if (to[u] >= 0 && hl == 7) kept[to[u]] = from[u];
                if (pf[u] >= 0 && pt[u] >= 0) ev_store(p, row[u], pt[u], to[u] % kPage, g, hl);
            }
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
        if (i0 == 0 || overlap) sync_cluster();
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
            const int i = i0 + half + u * halves;
            if (i < r && from[u] >= 0 && to[u] >= 0) ev_store(p, row[u], to[u], (p.keep - r + i) % kPage, g, hl);
        }
    }
}

__global__ void evict_done_kernel() {}  // an ordinary launch: it starts when the eviction has ended
