// qsa_prompt_attn.cuh -- causal attention over whole packed prompts on the tensor cores.
//
// Mathematics: for row i of a sequence's n query rows against its m key rows,
//   O_i = sum_{j <= i + m - n} exp(x_ij - M_i) V_j / sum_j exp(x_ij - M_i),  x_ij = scale * q_i . k_j,
// in one pass over the keys with a running reference maximum M and sum; both are fp32.
//
// One CTA computes 128 rows of one head:
//   * Q (128 x 256) stays in shared memory; K and V tiles of 128 keys stream through a ring of
//     five 32 KB slots (half a tile each) that one thread fills by TMA;
//   * one thread issues the tcgen05.mma: S_i = Q K_i^T into one of two 128-column TMEM buffers
//     (so S_{i+1} is computed while the softmax works on S_i), then O += P_i V_i with P_i read
//     from TMEM (the weights overwrite their scores as 16-bit pairs) and V_i as an MN-major
//     operand.  2 x 128 columns of S and 256 of O fill the 512 of TMEM;
//   * four softmax warps own a row per thread: no exchange between threads.  The reference
//     maximum moves only when a tile exceeds it by more than 2^8, so O is rarely rescaled.
//
// The weights are rounded to the input type for the tensor cores (fp16: 2^-12, bf16: 2^-9 relative, as
// the output is); the sum is over the unrounded weights in fp32.
//
// Every mbarrier wait is bounded and reports through the device status word.
#pragma once

#include "qsa_paged_cache.cuh"
#include "qsa_sm100.cuh"

namespace qsa {

constexpr int kFaM = 128;      // query rows of a CTA
constexpr int kFaN = 128;      // keys of a tile
constexpr int kFaSlots = 5;
constexpr int kFaSlotBytes = 32 * 1024;  // half a K or V tile
constexpr int kFaQBytes = kFaM * kD * 2;
constexpr int kFaThreads = 192;  // four softmax warps, TMA, MMA
constexpr float kFaShift = 8.f;
constexpr float kFaNoMax = -1.0e30f;

struct __align__(8) FaBarriers {
  uint64_t full[kFaSlots];
  uint64_t empty[kFaSlots];
  uint64_t q_full;
  uint64_t s_full[2];
  uint64_t p_ready[2];
  uint64_t pv_done;
  uint64_t tail;
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort;
};
constexpr int kFaSmemBytes = 1024 /*align*/ + kFaQBytes + kFaSlots * kFaSlotBytes + static_cast<int>(sizeof(FaBarriers));
static_assert(kFaSmemBytes <= 227 * 1024, "shared memory of a CTA");

struct FaArgs {
  const int* cu_q;
  const int* cu_k;
  int nseq;
  int rows_q, rows_k;
  int hq, group;
  float scale_log2;
  const void* gate;
  void* out;
  int64_t ldg, ldo;
  uint32_t* status;
};

// ---- TMEM and MMA forms this kernel needs beyond qsa_sm100.cuh

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// D (TMEM) (+)= A (TMEM) . B (shared memory)
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand with the 128-byte swizzle: rows of 64 MN elements (128 bytes), 8-row atoms
// `sbo` bytes apart along K, blocks of 64 MN elements `lbo` bytes apart.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16 instruction descriptor with both operands bf16 instead of fp16.
constexpr uint32_t kUmmaBf16 = (1u << 7) | (1u << 10);

// The sequence and 128-row block of flat tile `idx`, the last tile first (a sequence's last
// block sees the most keys, so the longest work starts first).  Every warp computes the same.
struct FaTile {
  int row0, rows;  // first packed query row of the tile; its rows (<= 0: no such tile)
  int key0, keys;  // first packed key row; keys that any row of the tile sees
  int seen0;       // keys that the tile's first row sees (row r sees seen0 + r)
};

__device__ __forceinline__ int fa_bound(const int* cu, int s, int rows) { return min(max(__ldg(cu + s), 0), rows); }

__device__ __forceinline__ FaTile fa_tile(const FaArgs& a, int idx) {
  const int lane = threadIdx.x & 31;
  FaTile t = {0, 0, 0, 0, 0};
  int total = 0;
  for (int s0 = 0; s0 < a.nseq; s0 += 32) {
    const int s = s0 + lane;
    if (s < a.nseq) total += (max(0, fa_bound(a.cu_q, s + 1, a.rows_q) - fa_bound(a.cu_q, s, a.rows_q)) + kFaM - 1) / kFaM;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (idx >= total) return t;
  const int want = total - 1 - idx;
  for (int s0 = 0, base = 0; s0 < a.nseq; s0 += 32) {
    const int s = s0 + lane;
    const int nb = s < a.nseq ? (max(0, fa_bound(a.cu_q, s + 1, a.rows_q) - fa_bound(a.cu_q, s, a.rows_q)) + kFaM - 1) / kFaM : 0;
    int inc = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + inc > want);
    if (past) {
      const int l = __ffs(past) - 1;
      const int seq = s0 + l, block = want - base - __shfl_sync(0xffffffffu, inc - nb, l);
      const int q0 = fa_bound(a.cu_q, seq, a.rows_q), n = fa_bound(a.cu_q, seq + 1, a.rows_q) - q0;
      const int k0 = fa_bound(a.cu_k, seq, a.rows_k), m = max(0, fa_bound(a.cu_k, seq + 1, a.rows_k) - k0);
      t.row0 = q0 + block * kFaM;
      t.rows = min(kFaM, n - block * kFaM);
      t.key0 = k0;
      t.seen0 = block * kFaM + 1 + m - n;
      t.keys = max(0, min(m, t.seen0 + t.rows - 1));
      return t;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  return t;
}

// grid: hq * (upper bound of the tiles), heads fastest (the heads of a KV head share its K and
// V through L2); block: 192; dynamic shared memory: kFaSmemBytes.
template <typename T>
__global__ void __launch_bounds__(kFaThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, FaArgs a) {
  constexpr uint32_t kType = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? kUmmaBf16 : 0u;
  constexpr uint32_t kIdescQK = umma_idesc_f16(kFaM, kFaN, false, false) | kType;
  constexpr uint32_t kIdescPV = umma_idesc_f16(kFaM, kD, false, true) | kType;
  extern __shared__ unsigned char fsm_raw[];
  unsigned char* fsm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(fsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* sq = fsm;
  unsigned char* ring = fsm + kFaQBytes;
  FaBarriers& fb = *reinterpret_cast<FaBarriers*>(ring + kFaSlots * kFaSlotBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = static_cast<int>(blockIdx.x) % a.hq, kvh = head / a.group;

  griddep_wait();
  const FaTile tile = fa_tile(a, static_cast<int>(blockIdx.x) / a.hq);
  if (tile.rows <= 0) return;
  const int ntiles = (tile.keys + kFaN - 1) / kFaN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFaSlots; ++s) {
      mbar_init(&fb.full[s], 1);
      mbar_init(&fb.empty[s], 1);
    }
    mbar_init(&fb.q_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&fb.s_full[b], 1);
      mbar_init(&fb.p_ready[b], 4);
    }
    mbar_init(&fb.pv_done, 1);
    mbar_init(&fb.tail, 1);
    mbar_init(&fb.drain, 1);
    fb.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 5) tmem_alloc(&fb.tmem_base, 512u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = fb.tmem_base;
  const uint32_t tmem_o = tmem + 2 * kFaN;

  if (warp == 4) {
    // ---------------- TMA: Q, then K_0, K_1, V_0, K_2, V_1, ...
    bool ok = true;
    if (lane == 0 && ntiles > 0) {
      mbar_expect_tx(&fb.q_full, kFaQBytes);
      for (int c = 0; c < 4; ++c) tma_load_3d(sq + c * (kFaM * 128), &tmap_q, 64 * c, head, tile.row0, &fb.q_full);
    }
    int n = 0;  // half tiles so far
    auto acquire = [&](int& slot) {
      slot = n % kFaSlots;
      const uint32_t parity = ((n / kFaSlots) & 1) ^ 1;
      ++n;
      return mbar_wait_warp(&fb.empty[slot], parity, &fb.abort, a.status);
    };
    auto load_k = [&](int i) {
      for (int h = 0; h < 2 && ok; ++h) {  // dims 128 h .. 128 h + 127 of 128 keys
        int slot;
        ok = acquire(slot);
        if (ok && lane == 0) {
          mbar_expect_tx(&fb.full[slot], kFaSlotBytes);
          for (int c = 0; c < 2; ++c)
            tma_load_3d(ring + slot * kFaSlotBytes + c * (kFaN * 128), &tmap_k, 64 * (2 * h + c), kvh,
                        tile.key0 + i * kFaN, &fb.full[slot]);
        }
      }
    };
    int tails = 0;
    auto load_v = [&](int i) {
      for (int h = 0; h < 2 && ok; ++h) {  // 64 keys, all dims
        int slot;
        ok = acquire(slot);
        if (!ok) return;
        unsigned char* dst = ring + slot * kFaSlotBytes;
        const int first = i * kFaN + 64 * h, valid = tile.keys - first;
        uint64_t* bar = valid >= 64 ? &fb.full[slot] : &fb.tail;
        if (lane == 0) {
          mbar_expect_tx(bar, kFaSlotBytes);
          for (int c = 0; c < 4; ++c) tma_load_3d(dst + c * (64 * 128), &tmap_v, 64 * c, kvh, tile.key0 + first, bar);
        }
        if (valid < 64) {
          // Rows behind the last key a row of this tile sees may be another sequence's, or
          // nobody's, and hold anything; a weight of 0 times NaN would spread, so they become 0.
          ok = mbar_wait_warp(&fb.tail, tails++ & 1, &fb.abort, a.status);
          if (!ok) return;
          const int r0 = max(valid, 0);
          for (int e = lane; e < (64 - r0) * 32; e += 32) {
            const int r = r0 + (e >> 5), c = (e >> 3) & 3, part = e & 7;
            *reinterpret_cast<uint4*>(dst + c * (64 * 128) + r * 128 + part * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&fb.full[slot]);
        }
      }
    };
    for (int i = 0; i < ntiles && ok; ++i) {
      load_k(i);
      if (i > 0 && ok) load_v(i - 1);
    }
    if (ntiles > 0 && ok) load_v(ntiles - 1);
    if (!ok && lane == 0) {  // drain copies that may still be in flight before the CTA leaves
      mbar_drain_wait(&fb.q_full, 0);
      if (tails > 0) mbar_drain_wait(&fb.tail, (tails - 1) & 1);
      for (int j = max(0, n - 1 - kFaSlots); j < n - 1; ++j) mbar_drain_wait(&fb.full[j % kFaSlots], (j / kFaSlots) & 1);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------- MMA
    if (lane == 0 && ntiles > 0) {
      int n = 0;
      bool ok = mbar_wait(&fb.q_full, 0, &fb.abort, a.status);
      const uint32_t q0 = smem_u32(sq), r0 = smem_u32(ring);
      auto take = [&](int& slot) {
        slot = n % kFaSlots;
        const uint32_t parity = (n / kFaSlots) & 1;
        ++n;
        const bool got = mbar_wait(&fb.full[slot], parity, &fb.abort, a.status);
        tc_fence_after();
        return got;
      };
      auto scores = [&](int i) {  // S_i = Q K_i^T
        for (int h = 0; h < 2 && ok; ++h) {
          int slot;
          if (!(ok = take(slot))) return;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = (ks >> 2) * (kFaM * 128) + (ks & 3) * 32;
            umma_f16(tmem + (i & 1) * kFaN, umma_desc_k_sw128(q0 + 2 * h * (kFaM * 128) + off, 1024),
                     umma_desc_k_sw128(r0 + slot * kFaSlotBytes + off, 1024), kIdescQK, h + ks > 0 ? 1u : 0u);
          }
          umma_commit(&fb.empty[slot]);
        }
        umma_commit(&fb.s_full[i & 1]);
      };
      if (ok) scores(0);
      for (int i = 0; i < ntiles && ok; ++i) {
        // S_{i+1} takes the buffer of P_{i-1}, which the product issued before has read
        if (i + 1 < ntiles) scores(i + 1);
        if (!ok || !(ok = mbar_wait(&fb.p_ready[i & 1], (i >> 1) & 1, &fb.abort, a.status))) break;
        tc_fence_after();
        for (int h = 0; h < 2 && ok; ++h) {  // O += P_i V_i
          int slot;
          if (!(ok = take(slot))) break;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ts(tmem_o, tmem + (i & 1) * kFaN + (h * 4 + ks) * 8,
                        umma_desc_mn_sw128(r0 + slot * kFaSlotBytes + ks * 2048, 64 * 128, 1024), kIdescPV,
                        i + h + ks > 0 ? 1u : 0u);
          umma_commit(&fb.empty[slot]);
        }
        if (ok) umma_commit(&fb.pv_done);
      }
      // every MMA this thread issued has completed once `drain` fires
      umma_commit(&fb.drain);
      mbar_drain_wait(&fb.drain, 0);
    }
    __syncwarp();
  } else {
    // ---------------- softmax: thread = row = TMEM lane
    const int r = warp * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int seen = tile.seen0 + r;  // keys this row sees
    float m_run = kFaNoMax, l_run = 0.f;
    bool ok = true;
    for (int i = 0; i < ntiles; ++i) {
      const uint32_t ts = tmem + lanes + (i & 1) * kFaN;
      if (!(ok = mbar_wait_warp(&fb.s_full[i & 1], (i >> 1) & 1, &fb.abort, a.status))) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
      tmem_ld_wait();
      const int left = seen - i * kFaN;  // columns below this are seen
      if (__any_sync(0xffffffffu, left < kFaN)) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= left) s[c] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[c + e]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
      if (__any_sync(0xffffffffu, top > m_run + kFaShift)) {
        // a row's own decision: its result does not depend on the other rows of the tile
        const float mnew = top > m_run + kFaShift ? top : m_run;
        const float alpha = exp2f(m_run - mnew);
        m_run = mnew;
        l_run *= alpha;
        if (i > 0) {  // O of this warp's rows, once P_{i-1} V_{i-1} is in
          if (!(ok = mbar_wait_warp(&fb.pv_done, (i - 1) & 1, &fb.abort, a.status))) break;
          tc_fence_after();
          for (int c = 0; c < kD; c += 32) {
            uint32_t o[32];
            tmem_ld32(tmem_o + lanes + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tmem_o + lanes + c, o);
          }
          tmem_st_wait();
        }
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 128; c += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(fmaf(__uint_as_float(s[c + e]), a.scale_log2, -m_run)));
          sum[e] += p;
          s[c + e] = __float_as_uint(p);
        }
        // the pair (c, c + 1) goes into word c / 2
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          s[c / 2] = pack_bf162(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          s[c / 2 + 1] = pack_bf162(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        } else {
          s[c / 2] = pack_half2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          s[c / 2 + 1] = pack_half2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        }
      }
      l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_st32(ts, s);
      tmem_st32(ts + 32, s + 32);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&fb.p_ready[i & 1]);
    }
    // ---------------- O / l, gated
    if (ok && ntiles > 0) ok = mbar_wait_warp(&fb.pv_done, (ntiles - 1) & 1, &fb.abort, a.status);
    if (ok) {
      tc_fence_after();
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      const bool mine = r < tile.rows;
      const int row = tile.row0 + r;
      T* dst = static_cast<T*>(a.out) + row * a.ldo + head * kD;
      const T* gsrc = a.gate ? static_cast<const T*>(a.gate) + row * a.ldg + head * kD : nullptr;
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (ntiles > 0) {
          tmem_ld32(tmem_o + lanes + c, o);
          tmem_ld_wait();
        }
        if (mine) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = l_run > 0.f ? __uint_as_float(o[8 * j + e]) * inv : 0.f;
            if (gsrc) {
              Row8<T> graw;
              graw.load(gsrc + c + 8 * j);
              float gv[8];
              graw.get(gv);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= gate_factor(gv[e]);
            }
            Row8<T>::store(dst + c + 8 * j, x);
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 512u);
}

}  // namespace qsa
