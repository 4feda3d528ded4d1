// Several query tokens per sequence over an fp8 cache, on the 5th-generation tensor cores: the
// step of multi_tc_kernel with its keys and values in fp8 blocks. The new tokens were quantised
// into their blocks by the kernel before (kv_append_fp8_kernel), so every key is read from the
// cache: query row (t, h) at position p = L - n + t attends the cached positions lo .. p.
//
// The codes are turned into fp16 operands in shared memory, their token's scale with them. A page
// (16 tokens) has a power of two 2^E at least as large as its K scales, 2^F for its V scales, and
//     K'_j = fp16(code_j ks_j 2^-E),   V'_j = fp16(code_j vs_j 2^-F):
// code times a factor in (0, 1], rounded once (2^-12 of the element, or of 2^-13 of the page's largest
// factor), nothing to overflow. 2^E goes into the page's score multiplier; 2^F into the exponent of
// its probabilities, so that the output accumulates in one unit:
//     s_j + F = (q K'_j) (scale log2(e) 2^E) + F,   P_j = fp16(2^(s_j + F - R + 7)),
//     O = sum P_j V'_j = 2^(7-R) sum 2^(s_j) v_j,   l = sum over pages 2^-F sum P_j = 2^(7-R) sum 2^(s_j)
// with R a running reference of s_j + F per row (the next integer, moved only when exceeded by more
// than 2^8, as in multi_tc_kernel): the probabilities stay below 2^15, and fp16 holds them to 2^-12 (to 2^-31 of the
// largest for the smallest ones). Multiplying the scores by their token's scale in the softmax
// instead would be exact, but every factor is then read from shared memory by every row: 4 bytes a
// lane and key, more than the whole softmax takes. Scales beyond 2^100 (K) or outside 2^-60 ..
// 2^60 (V) lose bits.
//
// One CTA per (sequence, KV head, block of 128 query rows, key split); 9 warps:
//   warps 0-3  one query row per thread (TMEM lane = row): the softmax and the finish
//   warps 4-7  warp 4 + u copies tile u of every 64-key block (one 2176-byte block, a bulk copy
//              into its own ring of raw blocks) and writes its K' and V' into the stage
//   warp 8     issues the MMAs: S_j = Q K'_j^T and O += P_j V'_j (V' as it is stored, transposed:
//              tokens contiguous, so both operands are K-major)
constexpr int kT8Rows = 128, kT8Keys = 64, kT8Tiles = kT8Keys / kPage;
#ifndef DA_T8_STAGES
#define DA_T8_STAGES 3
#endif
#ifndef DA_T8_RAW
#define DA_T8_RAW 4
#endif
constexpr int kT8Stages = DA_T8_STAGES;  // blocks of K' and V'
constexpr int kT8Raw = DA_T8_RAW;        // fp8 blocks in flight per copying warp
constexpr int kT8SBufs = 2;
constexpr int kT8HalfBytes = kT8Keys * kD * 2;  // 8 KiB of K' (or V')
constexpr int kT8StageBytes = 2 * kT8HalfBytes;
constexpr int kT8QBytes = kT8Rows * kD * 2;
constexpr int kT8RawBytes = kT8Tiles * kT8Raw * kBlk8Bytes;
constexpr int kT8Bars = kT8Tiles * kT8Raw + 2 * kT8Stages + 3 * kT8SBufs + 1;
constexpr int kT8Smem = 1024 + kT8QBytes + kT8Stages * kT8StageBytes + kT8RawBytes + kT8Stages * kT8Tiles * 16 + kT8Bars * 8;
constexpr int kT8Warps = 9, kT8Threads = kT8Warps * 32;
constexpr uint32_t kT8TmemCols = 256, kT8ColS = 0, kT8ColO = 64 * kT8SBufs;
constexpr float kT8Rescale = 8.f, kT8Shift = 7.f;  // log2: a row's reference may be exceeded by; the probabilities' unit
constexpr int kT8MaxE = 100, kT8MaxF = 60;

__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__global__ void __launch_bounds__(kT8Threads, 2)
    multi_tc8_kernel(const MultiParams p, const uint8_t *__restrict__ kv) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem;                    // [128 rows][128 B], 128-byte swizzle
    uint8_t *sKV = smem + kT8QBytes;       // [stage][K' block [64 tokens][128 B] | V' block [64 d][128 B]]
    uint8_t *sRaw = sKV + kT8Stages * kT8StageBytes;  // [tile][kT8Raw][2176]
    float4 *s_fac = reinterpret_cast<float4 *>(sRaw + kT8RawBytes);  // [stage][tile]: multiplier, F, 2^-F
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_fac + kT8Stages * kT8Tiles);
    const uint32_t raw_full = smem_addr(bars);  // [tile][kT8Raw]
    const uint32_t kv_full = raw_full + 8 * kT8Tiles * kT8Raw, kv_empty = kv_full + 8 * kT8Stages;
    const uint32_t s_full = kv_empty + 8 * kT8Stages, p_full = s_full + 8 * kT8SBufs;
    const uint32_t o_done = p_full + 8 * kT8SBufs, drain = o_done + 8 * kT8SBufs;
    __shared__ int s_page[kMMaxChunk];
    __shared__ __align__(16) uint32_t s_vfac[kT8Tiles][kPage];  // V factors: 16 high halves, then 16 low ones
    __shared__ uint32_t s_tmem;
    __shared__ int s_ticket;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int split = blockIdx.x % p.splits, rb = blockIdx.x / p.splits;
    const int g = blockIdx.y, b = blockIdx.z;

    if (tid == 0) {
        for (int s = 0; s < kT8Tiles * kT8Raw; ++s) mbar_init(raw_full + 8 * s, 1);
        for (int s = 0; s < kT8Stages; ++s) {
            mbar_init(kv_full + 8 * s, kT8Tiles);
            mbar_init(kv_empty + 8 * s, 1);
        }
        for (int s = 0; s < kT8SBufs; ++s) {
            mbar_init(s_full + 8 * s, 1);
            mbar_init(p_full + 8 * s, 4);  // the four row warps
            mbar_init(o_done + 8 * s, 1);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int W = p.window;
    const int r0 = rb * kT8Rows;
    const int r_end = min(r0 + kT8Rows, p.T * p.G);
    int key_lo, key_end;
    const MultiKeys keys = multi_keys_cached(p, b, r0, r_end, key_lo, key_end);
    if (keys.bad && tid == 0 && g == 0 && blockIdx.x == 0) flag_status(DA_STATUS_BAD_SEQ_LEN);
    const int n = keys.n, base = keys.base, pt_lo = keys.pt_lo, ntiles = keys.ntiles;
    const int kb = split * p.chunk;
    const int ke = min(kb + p.chunk, ntiles);
    const int nsplit = (ntiles + p.chunk - 1) / p.chunk;
    const size_t bg = static_cast<size_t>(b) * p.Hkv + g;
    auto row_off = [&](int r) {
        const int t = r / p.G, hl = r - t * p.G;
        return ((static_cast<size_t>(b) * p.T + t) * p.Hq + g * p.G + hl) * kD;
    };
    if (kb >= ke) {
        if (ntiles == 0 && split == 0)
            for (int i = tid; i < (r_end - r0) * (kD / 8); i += blockDim.x)
                *reinterpret_cast<uint4 *>(p.out + row_off(r0 + i / (kD / 8)) + (i % (kD / 8)) * 8) =
                    make_uint4(0, 0, 0, 0);
        return;
    }
    const int cnt = ke - kb;
    const int nblk = (cnt + kT8Tiles - 1) / kT8Tiles;
    const int r_valid = min(r_end, r0 + max(0, n * p.G - r0));  // rows r0 .. r_valid-1 are queries

    // ---- page indices, query rows as fp16 (zero past the valid ones), TMEM
    for (int i = tid; i < cnt; i += blockDim.x) {
        int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + pt_lo + kb + i);
        if (page < 0 || page >= p.num_pages) {
            flag_status(DA_STATUS_BAD_PAGE);
            page = -1;  // its tokens read as zeros
        }
        s_page[i] = page;
    }
    if (warp < 4) {
        const int r = r0 + tid;
        const bool ok = r < r_valid;
        const uint4 *src = ok ? reinterpret_cast<const uint4 *>(p.q + row_off(r)) : nullptr;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint4 v = ok ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            v = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
            *reinterpret_cast<uint4 *>(sQ + tid * 128 + ((c ^ (tid & 7)) << 4)) = v;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q is read by the tensor cores
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(kT8TmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    bool failed = false;
    if (warp >= 4 && warp < 8) {
        // ---- copies and operands: tile u of every block
        const int u = warp - 4;
        uint8_t *raw = sRaw + u * kT8Raw * kBlk8Bytes;
        const uint32_t full0 = raw_full + 8 * u * kT8Raw;
        const uint64_t policy = evict_first_policy();
        const int mine = cnt > u ? (cnt - u + kT8Tiles - 1) / kT8Tiles : 0;  // blocks whose tile u exists
        auto issue = [&](int j) {  // (lane 0)
            const int page = s_page[j * kT8Tiles + u], s = j % kT8Raw;
            const uint32_t bar = full0 + 8 * s;
            if (page < 0) {  // nothing to copy: the phase completes by itself
                mbar_arrive(bar);
                return;
            }
            mbar_expect_tx(bar, kBlk8Bytes);
            const uint8_t *src = kv + (static_cast<size_t>(page) * p.Hkv + g) * kBlk8Bytes;
            if (p.row_blocks == 1)
                bulk_load_hint(smem_addr(raw + s * kBlk8Bytes), src, kBlk8Bytes, bar, policy);
            else  // other row blocks read it too
                bulk_load(smem_addr(raw + s * kBlk8Bytes), src, kBlk8Bytes, bar);
        };
        int issued = 0;
        if (lane == 0)
            for (; issued < mine && issued < kT8Raw; ++issued) issue(issued);
        for (int j = 0; j < nblk; ++j) {
            const int st = j % kT8Stages;
            uint4 kc[2], vc[2];
            float sc = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
            if (j < mine) {
                if (__any_sync(0xffffffffu, !mbar_wait_bounded(full0 + 8 * (j % kT8Raw), (j / kT8Raw) & 1))) {
                    failed = true;
                    break;
                }
                const int k = j * kT8Tiles + u;
                if (s_page[k] >= 0) {
                    const uint8_t *blk = raw + (j % kT8Raw) * kBlk8Bytes;
                    const int pos0 = (pt_lo + kb + k) * kPage;
                    // a token outside the rows' keys may hold anything: its codes and scales are zeros
                    auto key = [&](int t) { return pos0 + t >= key_lo && pos0 + t < key_end; };
                    if (key(lane & 15)) sc = reinterpret_cast<const float *>(blk + kBlk8S)[lane];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (key((lane >> 2) + 8 * i)) kc[i] = reinterpret_cast<const uint4 *>(blk)[lane + 32 * i];
                        vc[i] = reinterpret_cast<const uint4 *>(blk + kBlk8V)[lane + 32 * i];
                    }
                    if (pos0 < key_lo || pos0 + kPage > key_end) {  // (V rows hold the 16 tokens' bytes)
                        uint32_t m[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            m[e] = (key(4 * e) ? 0xffu : 0u) | (key(4 * e + 1) ? 0xff00u : 0u) |
                                   (key(4 * e + 2) ? 0xff0000u : 0u) | (key(4 * e + 3) ? 0xff000000u : 0u);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            vc[i] = make_uint4(vc[i].x & m[0], vc[i].y & m[1], vc[i].z & m[2], vc[i].w & m[3]);
                    }
                }
            }
            // the page's powers of two, and each token's factor as two fp16 values (K: lanes 0-15, V: 16-31)
            float top = fabsf(sc);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const int lim = lane < 16 ? kT8MaxE : kT8MaxF;
            const int ex = max(-lim, min(lim, static_cast<int>(__float_as_uint(top) >> 23) - 126));
            const float fac = sc * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            const __half hi = __float2half_rn(fac), lo = __float2half_rn(fac - __half2float(hi));
            uint32_t packed = static_cast<uint32_t>(__half_as_ushort(hi)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
            __syncwarp();  // the raw block and the previous block's V factors have been read
            if (lane >= 16) {
                unsigned short *f = reinterpret_cast<unsigned short *>(s_vfac[u]);
                f[lane - 16] = __half_as_ushort(hi);
                f[lane] = __half_as_ushort(lo);
            }
            if (lane == 0 && issued < mine) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                issue(issued);
                ++issued;
            }
            __syncwarp();
            if (j >= kT8Stages && __any_sync(0xffffffffu, !mbar_wait_bounded(kv_empty + 8 * st, ((j / kT8Stages) - 1) & 1))) {
                failed = true;
                break;
            }
            float *fo = reinterpret_cast<float *>(s_fac + st * kT8Tiles + u);
            if (lane == 0) fo[0] = fmaxf(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23), 1.1754944e-38f);
            if (lane == 16) {
                fo[1] = static_cast<float>(ex);
                fo[2] = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            }
            uint8_t *sK = sKV + st * kT8StageBytes, *sV = sK + kT8HalfBytes;
            const uint4 *vf = reinterpret_cast<const uint4 *>(s_vfac[u]);
            const uint4 f0 = vf[0], f1 = vf[1], f2 = vf[2], f3 = vf[3];
            const uint32_t vh[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
            const uint32_t vl[8] = {f2.x, f2.y, f2.z, f2.w, f3.x, f3.y, f3.z, f3.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                {  // K: token (lane / 4) + 8 i, elements 16 (lane % 4) .. + 15
                    const int t = (lane >> 2) + 8 * i, row = u * kPage + t;
                    const uint32_t f = __shfl_sync(0xffffffffu, packed, t);
                    const uint32_t fh = __byte_perm(f, f, 0x1010), fl = __byte_perm(f, f, 0x3232);
                    const uint32_t w[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a, c;
                        e4m3x4_to_f16x2x2(w[e], a, c);
                        o[2 * e] = hfma2(a, fh, hmul2(a, fl));
                        o[2 * e + 1] = hfma2(c, fh, hmul2(c, fl));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<uint4 *>(sK + row * 128 + (((2 * (lane & 3) + h) ^ (row & 7)) << 4)) =
                            make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
                }
                {  // V: element d = lane + 32 i, the tile's 16 tokens
                    const int d = lane + 32 * i;
                    const uint32_t w[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a, c;
                        e4m3x4_to_f16x2x2(w[e], a, c);
                        o[2 * e] = hfma2(a, vh[2 * e], hmul2(a, vl[2 * e]));
                        o[2 * e + 1] = hfma2(c, vh[2 * e + 1], hmul2(c, vl[2 * e + 1]));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<uint4 *>(sV + d * 128 + (((2 * u + h) ^ (d & 7)) << 4)) =
                            make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full + 8 * st);
        }
        if (lane == 0 && failed)  // nothing may still be landing when the CTA leaves
            for (int j = max(0, issued - kT8Raw); j < issued; ++j) mbar_wait_idle(full0 + 8 * (j % kT8Raw), (j / kT8Raw) & 1);
        __syncwarp();
    } else if (warp == 8) {
        // ---- MMA issuer: S_j = Q K'_j^T, then O += P_{j-1} V'_{j-1}
        const bool leader = elect_one();
        const uint32_t id_qk = umma_idesc_f16(kT8Rows, kT8Keys), id_pv = umma_idesc_f16(kT8Rows, kD);
        const uint64_t dq = umma_sdesc(smem_addr(sQ), 16, 1024), dk = umma_sdesc(smem_addr(sKV), 16, 1024);
        const uint64_t dv = umma_sdesc(smem_addr(sKV) + kT8HalfBytes, 16, 1024);
        auto wait_all = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_idle(bar, parity)); };
        auto scores = [&](int j) {
            const int s = j % kT8Stages, sb = j % kT8SBufs;
            if (!wait_all(kv_full + 8 * s, (j / kT8Stages) & 1) ||
                (j >= kT8SBufs && !wait_all(o_done + 8 * sb, ((j / kT8SBufs) - 1) & 1)))
                return false;
            tc_fence_after();
            const uint64_t dks = dk + s * (kT8StageBytes / 16);
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    umma_bf16_ss(tm + kT8ColS + 64 * sb, dq + 2 * kk, dks + 2 * kk, id_qk, kk > 0);
                umma_commit(s_full + 8 * sb);
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int jj) {
            const int s = jj % kT8Stages, pb = jj % kT8SBufs;
            if (!wait_all(p_full + 8 * pb, (jj / kT8SBufs) & 1)) return false;
            tc_fence_after();
            const uint64_t dvs = dv + s * (kT8StageBytes / 16);
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < kT8Keys / 16; ++kk)
                    umma_bf16_ts(tm + kT8ColO, tm + kT8ColS + 64 * pb + 8 * kk, dvs + 2 * kk, id_pv, kk > 0 || jj > 0 ? 1u : 0u);
                umma_commit(o_done + 8 * pb);
                umma_commit(kv_empty + 8 * s);
            }
            __syncwarp();
            return true;
        };
        for (int j = 0; j <= nblk && !failed; ++j)
            if ((j < nblk && !scores(j)) || (j >= 1 && !values(j - 1))) failed = true;
        if (leader) {
            umma_commit(drain);  // completes when every MMA issued above has
            mbar_wait_bounded(drain, 0);
        }
        __syncwarp();
    } else {
        // ---- query rows: one per thread
        const int r = r0 + tid;
        const bool valid = r < r_valid;
        const bool warp_active = r0 + 32 * warp < r_valid;
        const int t = r / p.G;
        const int pr = valid ? base + t : -1;
        const int lor = valid && W > 0 ? max(0, base + t - W + 1) : 0;
        const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
        float m_ref = -INFINITY, l = 0.f;
        for (int j = 0; j < nblk; ++j) {
            const int k0 = kb + j * kT8Tiles;
            // every row warp waits for S_j, rows or not, so that no warp's arrival on p_full can run ahead
            // into a later phase (a give-up is taken by the whole warp: the TMEM accesses are warp-wide)
            const int sb = j % kT8SBufs, st = j % kT8Stages;
            if (__any_sync(0xffffffffu, !mbar_wait_bounded(s_full + 8 * sb, (j / kT8SBufs) & 1))) {
                failed = true;
                break;
            }
            if (warp_active) {
                // the pages' factors: complete since S_j is, waited for to see them (the stage is not
                // filled again before this block's P)
                if (__any_sync(0xffffffffu, !mbar_wait_bounded(kv_full + 8 * st, (j / kT8Stages) & 1))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const uint32_t sc = tm + lanes + kT8ColS + 64 * sb;
                uint32_t raw[2][32];
                tmem_ld32(sc, raw[0]);
                tmem_ld32(sc + 32, raw[1]);
                tmem_wait_ld();
                float x[64];
#pragma unroll
                for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(raw[c >> 5][c & 31]);
                const int jf = (pt_lo + k0) * kPage;
                if (!(valid && k0 + kT8Tiles <= ke && jf >= lor && jf + kT8Keys - 1 <= pr)) {
                    // keys [a, e) of the block are this row's
                    const int a = lor - jf, e = min(pr + 1 - jf, (ke - k0) * kPage);
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c < a || c >= e) x[c] = -INFINITY;
                }
                float4 fac[kT8Tiles];
                float mb = -INFINITY;
#pragma unroll
                for (int u = 0; u < kT8Tiles; ++u) {
                    fac[u] = s_fac[st * kT8Tiles + u];
                    const float *y = x + 16 * u;
                    const float m1 = max3(y[0], y[1], y[2]), m2 = max3(y[3], y[4], y[5]), m3 = max3(y[6], y[7], y[8]);
                    const float m4 = max3(y[9], y[10], y[11]), m5 = max3(y[12], y[13], y[14]);
                    const float mt = max3(max3(m1, m2, m3), max3(m4, m5, y[15]), -INFINITY);
                    mb = fmaxf(mb, fmaf(mt, fac[u].x, fac[u].y));  // the multiplier is positive
                }
                const bool need = valid && mb > m_ref + kT8Rescale;
                const float m_new = need ? ceilf(mb) : m_ref;  // an integer: F - R and the rescaling are exact
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    const int jb = (j - 1) % kT8SBufs;  // (see multi_tc_kernel on this wait)
                    if (__any_sync(0xffffffffu, !mbar_wait_bounded(o_done + 8 * jb, ((j - 1) / kT8SBufs) & 1))) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const float f = need ? exp2f(m_ref - m_new) : 1.f;  // m_ref = -inf: 0 (O and l are 0)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {  // (16 columns at a time: the 64 scores hold most registers)
                        uint32_t o[16];
                        tmem_ld16(tm + lanes + kT8ColO + 16 * h, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                        tmem_st16(tm + lanes + kT8ColO + 16 * h, o);
                        tmem_wait_st();
                    }
                }
                if (need) {
                    l *= exp2f(m_ref - m_new);
                    m_ref = m_new;
                }
                const float mr = kT8Shift - (m_ref == -INFINITY ? 0.f : m_ref);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int u = 2 * h + v;
                        const float2 mul = make_float2(fac[u].x, fac[u].x), add = make_float2(fac[u].y + mr, fac[u].y + mr);
                        float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float2 a = fma2(make_float2(x[16 * u + 2 * c], x[16 * u + 2 * c + 1]), mul, add);
                            const float a0 = fast_exp2(a.x), a1 = fast_exp2(a.y);
                            ls[c & 1] = add2(ls[c & 1], make_float2(a0, a1));
                            pk[8 * v + c] = pack_f16(a0, a1);
                        }
                        l += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) * fac[u].z;
                    }
                    tmem_st16(tm + lanes + kT8ColS + 64 * sb + 16 * h, pk);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 8 * sb);
        }
        // ---- finish this thread's row: O (after the last PV) -> output or partial
        const int lb = (nblk - 1) % kT8SBufs;
        if (warp_active && !failed && __any_sync(0xffffffffu, !mbar_wait_bounded(o_done + 8 * lb, ((nblk - 1) / kT8SBufs) & 1)))
            failed = true;
        const bool have = warp_active && !failed;
        const float m_row = m_ref - kT8Shift;
        float f = 0.f;  // rows that are not queries: zeros
        if (nsplit == 1 && valid && have) {
            const int h = g * p.G + (r - t * p.G);
            const float sg = p.sinks != nullptr ? __ldg(p.sinks + h) * kLog2e : -INFINITY;
            const float M = fmaxf(m_row, sg);
            if (M != -INFINITY) {
                const float den = l * exp2f(m_row - M) + (sg == -INFINITY ? 0.f : exp2f(sg - M));
                f = den > 0.f ? exp2f(m_row - M) / den : 0.f;
            }
        }
        float *slot = p.part + ((((bg * p.row_blocks + rb) * p.splits + split) * kT8Rows) + tid) * kMSlotFloats;
        if (nsplit > 1 && r < r_valid) {
            slot[0] = m_row;
            slot[1] = l;
        }
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t raw[16];
            if (have) {  // (the whole warp)
                tmem_ld16(tm + lanes + kT8ColO + 16 * h, raw);
                tmem_wait_ld();
            }
            float o[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = have && valid ? __uint_as_float(raw[c]) : 0.f;
            if (nsplit == 1) {
                if (r < r_end) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + row_off(r)) + 2 * h;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint4 w;
                        w.x = pack_bf16(o[8 * c] * f, o[8 * c + 1] * f);
                        w.y = pack_bf16(o[8 * c + 2] * f, o[8 * c + 3] * f);
                        w.z = pack_bf16(o[8 * c + 4] * f, o[8 * c + 5] * f);
                        w.w = pack_bf16(o[8 * c + 6] * f, o[8 * c + 7] * f);
                        dst[c] = w;
                    }
                }
            } else if (r < r_valid) {
                float4 *acc = reinterpret_cast<float4 *>(slot + kMAccOff) + 4 * h;
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            }
        }
    }
    if (failed) flag_status(DA_STATUS_TIMEOUT);

    // ---- teardown: every MMA done (the issuer has waited) before TMEM is released
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kT8TmemCols));
    }
    if (nsplit == 1 || p.defer) return;  // p.defer: multi_combine_kernel follows
    __threadfence();
    __syncthreads();
    int *ctr = p.counters + bg * p.row_blocks + rb;
    if (tid == 0) s_ticket = atomicAdd(ctr, 1);
    __syncthreads();
    if (s_ticket != nsplit - 1) return;
    __threadfence();
    const size_t slot0 = ((bg * p.row_blocks + rb) * p.splits) * static_cast<size_t>(kT8Rows);
    multi_combine_rows(p, p.part + slot0 * kMSlotFloats, kT8Rows, r0, r_end, n, b, g, nsplit, 0, kT8Rows, warp,
                       kT8Warps, lane);
    __syncthreads();
    if (tid == 0) *ctr = 0;  // ready for the next call
}
