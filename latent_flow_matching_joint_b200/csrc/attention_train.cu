// Attention for training: the forward pass with its row statistics, and the
// backward pass, which recomputes the probabilities from them.
//
//   forward   S = scale Q K^T,  P = softmax(S),  O = P V,  lse = log sum exp(S)
//   backward  D = rowsum(dO o O),  P = exp(S - lse),  dV = P^T dO,
//             dS = P o (dO V^T - D),  dQ = scale dS K,  dK = scale dS^T Q
//
// Queries, keys and values are rows of the same sequence, any strides, query
// heads sharing key heads in groups. A batch item's text may be padded: rows
// [txt_len, n_txt) then neither attend nor are attended to, whatever they
// hold. The sequence is cut into slots of 128 rows, text and the rows after
// it separately, so in every slot the rows in use come first; a slot without
// any is skipped.
//
// Rows past a slot's last row in use are masked: in the scores (a select, not
// an addition, so that nothing they hold gets through), and, where such a row
// is summed over by a product, by zeroing it in shared memory before the
// tensor core reads the tile (0 x NaN is NaN). Only a text's last slot
// needs that; past the end of the sequence TMA fills with zeros by itself.
//
// Tiles [128 rows][128 d] are loaded once and read by the tensor core both
// ways: contiguous along the contraction (scores) and across it (the
// products with V, dO, Q and K), by the operand descriptors alone.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace klein {

namespace {

constexpr int kAtTile = 128 * 128 * 2;   // 128 rows x 128 d, bf16: two boxes of 64 d, 16 KB each
constexpr int kAtBox = kAtTile / 2;
constexpr int kAtThreads = 320;
constexpr uint32_t kAtTmem = 512;
constexpr float kAtRescale = 8.0f;       // log2 units: the running maximum moves only when a row's maximum grows by > 2^8
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kFwdBar = 6 * kAtTile;     // 2 query tiles, 2 stages of K, 2 of V
constexpr int kFwdSmem = kFwdBar + 256 + 1024;

constexpr int kBwdWarps = 16;                      // elementwise warps of the backward kernel (8: 2 % slower)
constexpr int kBwdThreads = 64 + 32 * kBwdWarps;
constexpr int kBwdCols = 128 / (kBwdWarps / 4);    // columns of a tile per warp
static_assert(kBwdCols == 32, "a warp's columns are one tensor-memory load");
// Shared memory: 2 resident tiles, a ring of 3 of the first streamed tile (it
// is needed from the scores to the end of its step, and the next step's scores
// are made half a step ahead), a ring of 2 of the second, with the statistics.
constexpr int kBwdRingS = 2 * kAtTile;
constexpr int kBwdRingT = 5 * kAtTile;
constexpr int kBwdStat = 7 * kAtTile;
constexpr int kStatBytes = 2 * 128 * 4;
constexpr int kBwdBar = kBwdStat + 2 * kStatBytes;
constexpr int kBwdSmem = kBwdBar + 256;
static_assert(kBwdSmem <= 227 * 1024, "shared memory of one CTA");

// 16 rows of a tile as the contraction (d, the contiguous index, is the operand's own).
__device__ __forceinline__ uint64_t across_desc(uint32_t saddr) { return sw128_desc_mn(saddr, kAtBox); }

constexpr uint32_t kIdescAlong = idesc_bf16_f32(128, 128);
constexpr uint32_t kIdescAcross = kIdescAlong | (1u << 16);  // B is contiguous along its own index

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tile_load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int head, int b) {
  tma_load_4d(dst, map, bar, 0, row, head, b);
  tma_load_4d(dst + kAtBox, map, bar, 64, row, head, b);
}

// Zeroes rows [valid, 128) of a tile; the whole warp takes part.
__device__ __forceinline__ void scrub_rows(uint8_t* tile, int valid, int lane) {
  const int chunks = (128 - valid) * 8;  // 16-byte pieces of one box
  for (int i = lane; i < 2 * chunks; i += 32) {
    const int box = i >= chunks;
    *reinterpret_cast<uint4*>(tile + box * kAtBox + valid * 128 + (i - box * chunks) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
  __syncwarp();
}

// The slots of one batch item.
struct Slots {
  int rows, n_txt, txt_slots, slots, len;
  __device__ __forceinline__ Slots(const AttnTrainArgs& a, int b) {
    rows = a.rows;
    n_txt = a.n_txt;
    txt_slots = (a.n_txt + 127) >> 7;
    slots = a.slots;
    len = 0;
    if (a.txt_len) {
      len = a.txt_len[b];  // (a plain load: the kernel before this one may have written it, see pdl_wait)
      len = len < 0 ? 0 : (len > n_txt ? n_txt : len);
    }
  }
  __device__ __forceinline__ int start(int s) const { return s < txt_slots ? s << 7 : n_txt + ((s - txt_slots) << 7); }
  // rows that the slot owns, and how many of them, from its start, are in use
  __device__ __forceinline__ int extent(int s) const {
    const int left = (s < txt_slots ? n_txt : rows) - start(s);
    return left > 128 ? 128 : (left < 0 ? 0 : left);
  }
  __device__ __forceinline__ int valid(int s) const {
    if (s >= txt_slots) return extent(s);
    const int left = len - start(s);
    return left > 128 ? 128 : (left < 0 ? 0 : left);
  }
  // the slots with rows in use, in order
  __device__ __forceinline__ int used() const { return ((len + 127) >> 7) + slots - txt_slots; }
  __device__ __forceinline__ int used_slot(int j) const {
    const int t = (len + 127) >> 7;
    return j < t ? j : txt_slots + j - t;
  }
  // Whether rows past the slot's rows in use hold something else (not TMA's zeros).
  __device__ __forceinline__ bool ragged(int s) const { return valid(s) < 128 && start(s) + valid(s) < rows; }
};

// D[128 x 128] (+)= A[128 x 128] B[128 x 128]^T: both tiles contiguous along
// the contraction (d).
__device__ __forceinline__ void mma_along(uint32_t d_tmem, const uint8_t* a, const uint8_t* b) {
  const uint64_t da = sw128_desc(smem_u32(a)), db = sw128_desc(smem_u32(b));
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * kAtBox + (kk & 3) * 32) >> 4;  // in the descriptors' 16-byte units
    umma_bf16_warp(d_tmem, da + off, db + off, kIdescAlong, kk != 0);
  }
}

// D[128 x 128 d] (+)= A B over half of the contraction (64 rows of the tile B):
// A in TMEM as packed bf16 from column a_tmem on.
__device__ __forceinline__ void mma_across_half(uint32_t d_tmem, uint32_t a_tmem, const uint8_t* b, int half,
                                                bool accumulate) {
  const uint64_t db = across_desc(smem_u32(b) + half * 4 * 2048);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    umma_bf16_tmem_a_warp(d_tmem, a_tmem + kk * 8, db + kk * (2048 >> 4), kIdescAcross, accumulate || kk != 0);
}

// The whole contraction, A as the backward kernel's warps leave it: each
// kBwdCols columns' packed values at the start of those columns.
__device__ __forceinline__ void mma_across_bwd(uint32_t d_tmem, uint32_t a_tmem, const uint8_t* b, bool accumulate) {
  const uint64_t db = across_desc(smem_u32(b));
  constexpr int kSteps = kBwdCols / 16;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    umma_bf16_tmem_a_warp(d_tmem, a_tmem + (kk / kSteps) * kBwdCols + (kk % kSteps) * 8, db + kk * (2048 >> 4),
                          kIdescAcross, accumulate || kk != 0);
}

__device__ __forceinline__ __nv_bfloat16* head_row(const HeadsView& v, int b, int head, int row) {
  return static_cast<__nv_bfloat16*>(v.data) + b * v.batch_stride + head * v.head_stride + row * v.row_stride;
}

// Sum of the products of eight bf16 pairs.
__device__ __forceinline__ float dot8(uint4 x, uint4 y) {
  const uint32_t xu[4] = {x.x, x.y, x.z, x.w}, yu[4] = {y.x, y.y, y.z, y.w};
  float d = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 a = unpack_bf16(xu[c]), b = unpack_bf16(yu[c]);
    d = fmaf(a.x, b.x, fmaf(a.y, b.y, d));
  }
  return d;
}

constexpr int kStatKeys = 16;

}  // namespace

// Forward. One CTA = two query slots (a, b) of one head, sharing every K/V
// tile; roles and pipeline as in the denoiser's attention kernel (320 threads:
// warp 0 TMA, warp 1 MMA, warps 2..5 and 6..9 the softmax of slot a and b, one
// query row per thread; P written over S in tensor memory and fed from there).
// Bound by each row's chain of scores, maximum, exponentials and P: the tensor
// pipe and the MUFU are both 61 % busy. 24 heads, 4608 rows: 210 us in short
// bursts (1240 TFLOP/s).
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_train_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const AttnTrainArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sm_q = smem;
  uint8_t* sm_k = smem + 2 * kAtTile;
  uint8_t* sm_v = smem + 4 * kAtTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFwdBar);
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;    // [2]
  uint64_t* v_full = bars + 3;    // [2]
  uint64_t* kv_empty = bars + 5;  // [2]
  uint64_t* s_full = bars + 7;    // [2 slots]: scores ready (phase j), final output ready (phase n)
  uint64_t* p_full = bars + 9;    // [2 slots][2 halves of the keys]
  uint64_t* drain = bars + 13;
  uint64_t* scrub = bars + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y;
  const int kv_head = head / (a.heads / a.kv_heads);
  const int b = blockIdx.z;

  if (warp == 0 && lane == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[2 * s], 128);
      mbar_init(&p_full[2 * s + 1], 128);
    }
    mbar_init(drain, 1);
    mbar_init(scrub, 1);
    fence_barrier_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kAtTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();  // inputs and outputs are touched only after the previous kernel completes

  const Slots seq(a, b);
  const int slot0 = blockIdx.x * 2;
  // keys to go through; none when neither slot has a row in use
  const int n = seq.valid(slot0) + seq.valid(slot0 + 1) > 0 ? seq.used() : 0;

  if (warp == 0) {
    if (n > 0) {
      StageLog klog, vlog;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, 2 * kAtTile);
        for (int t = 0; t < 2; ++t) tile_load(sm_q + t * kAtTile, &map_q, q_full, seq.start(slot0 + t), head, b);
      }
      int scrubs = 0;
      for (int j = 0; j < n; ++j) {
        const int st = j & 1;
        const int slot = seq.used_slot(j), row = seq.start(slot);
        if (!mbar_wait_warp(&kv_empty[st], ((j >> 1) & 1) ^ 1, 0x401)) break;
        const bool ragged = seq.ragged(slot);
        if (lane == 0) {
          mbar_arrive_expect_tx(&k_full[st], kAtTile);
          klog.armed(st, (j >> 1) & 1);
          tile_load(sm_k + st * kAtTile, &map_k, &k_full[st], row, kv_head, b);
          mbar_arrive_expect_tx(ragged ? scrub : &v_full[st], kAtTile);
          if (!ragged) vlog.armed(st, (j >> 1) & 1);
          tile_load(sm_v + st * kAtTile, &map_v, ragged ? scrub : &v_full[st], row, kv_head, b);
        }
        if (ragged) {  // V rows that no query may see: P is 0 there, and so must they be
          __syncwarp();
          if (!mbar_wait_warp(scrub, scrubs & 1, 0x40b)) break;
          ++scrubs;
          scrub_rows(sm_v + st * kAtTile, seq.valid(slot), lane);
          if (lane == 0) {
            mbar_arrive(&v_full[st]);
            vlog.armed(st, (j >> 1) & 1);  // the log holds each stage's latest phase
          }
        }
        __syncwarp();
      }
      // no TMA write may land in shared memory after the CTA exits
      if (lane == 0 && mbar_wait(q_full, 0, 0x409)) {
        klog.drain(k_full, 2, 0x409);
        vlog.drain(v_full, 2, 0x409);
      }
    }
  } else if (warp == 1) {
    if (n > 0) {  // the whole warp, see umma_bf16_warp
      auto issue_s = [&](int t, int j) {
        mma_along(tmem_base + t * 256, sm_q + t * kAtTile, sm_k + (j & 1) * kAtTile);
        umma_commit_warp(&s_full[t]);
      };
      bool ok = mbar_wait_warp(q_full, 0, 0x402) && mbar_wait_warp(&k_full[0], 0, 0x403);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        issue_s(1, 0);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int st = j & 1;
        for (int t = 0; t < 2 && ok; ++t) {
          if (t == 0 && !mbar_wait_warp(&v_full[st], (j >> 1) & 1, 0x405)) { ok = false; break; }
          for (int half = 0; half < 2; ++half) {
            if (!mbar_wait_warp(&p_full[2 * t + half], j & 1, 0x404)) { ok = false; break; }
            tc_fence_after();
            mma_across_half(tmem_base + t * 256 + 128, tmem_base + t * 256 + half * 32, sm_v + st * kAtTile, half,
                            (j | half) != 0);
          }
          if (!ok) break;
          if (t == 1) umma_commit_warp(&kv_empty[st]);
          if (j + 1 < n) {
            if (t == 0) {
              if (!mbar_wait_warp(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, 0x406)) { ok = false; break; }
              tc_fence_after();
            }
            issue_s(t, j + 1);
          } else {
            umma_commit_warp(&s_full[t]);  // output of slot t final
          }
        }
      }
      // every MMA issued here has completed before TMEM is freed
      umma_commit_warp(drain);
      mbar_wait_warp(drain, 0, 0x40a);
    }
  } else {
    const int t = (warp - 2) >> 2;         // query slot of this warpgroup
    const int quarter = warp & 3;          // TMEM lane quarter of this warp
    const int rloc = quarter * 32 + lane;
    const int slot = slot0 + t;
    const int row = seq.start(slot) + rloc;
    const uint32_t s_col = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + t * 256;
    const uint32_t o_col = s_col + 128;
    const float sl2 = a.scale_log2;
    float m_run = -INFINITY;
    float l_run = 0.f;
    float s[128];
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp(&s_full[t], j & 1, 0x407)) { ok = false; break; }
      tc_fence_after();
      tmem_ld128(s_col, s);
      const int lim = seq.valid(seq.used_slot(j));
      if (lim < 128) {
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = (i < lim) ? s[i] : -INFINITY;
      }
      float m8[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) m8[q] = fmax3(s[q], s[q + 8], s[q + 16]);
#pragma unroll
      for (int i = 24; i < 120; i += 16) {
#pragma unroll
        for (int q = 0; q < 8; ++q) m8[q] = fmax3(m8[q], s[i + q], s[i + 8 + q]);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) m8[q] = fmaxf(m8[q], s[120 + q]);
      const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], fmax3(m8[5], m8[6], m8[7])));
      const float m_cand = mx * sl2;
      const bool grow = m_cand > m_run + kAtRescale;
      const float m_new = grow ? m_cand : m_run;
      // while every score of the row has been -inf, exponents are taken against 0
      const float m_sub = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = fast_exp2(m_run - m_sub);
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t pk[32];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 64 * half; i < 64 * half + 64; i += 2) {  // masked keys: exp2(-inf) = 0 exactly
          float x0, x1;
          ffma2(x0, x1, s[i], s[i + 1], sl2, sl2, -m_sub, -m_sub);
          const float p0 = fast_exp2(x0);
          const float p1 = fast_exp2(x1);
          fadd2(sa[(i >> 1) & 3], sb[(i >> 1) & 3], p0, p1);
          pk[(i >> 1) & 31] = pack_bf16(p0, p1);
        }
        if (half == 0 && j > 0 && __any_sync(0xffffffffu, grow)) {
          float o[32];
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(o_col + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(o_col + 32 * c, o);
          }
        }
        tmem_st32(s_col + 32 * half, reinterpret_cast<const float*>(pk));
        tc_fence_before();
        mbar_arrive(&p_full[2 * t + half]);
      }
      float sum4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) sum4[q] = sa[q] + sb[q];
      l_run = l_run * alpha + ((sum4[0] + sum4[1]) + (sum4[2] + sum4[3]));
      m_run = m_new;
    }
    const int valid = n > 0 ? seq.valid(slot) : 0;
    const bool own = rloc < seq.extent(slot);
    if (ok && (n == 0 || mbar_wait_warp(&s_full[t], n & 1, 0x408))) {
      tc_fence_after();
      // The warp's 32 rows leave through shared memory (K's ring: every score
      // has been made), so that whole rows of 256 bytes are written.
      const float inv = 1.0f / l_run;
      uint8_t* rows32 = sm_k + t * kAtTile + quarter * 32 * 256;
      if (n > 0) {
        float o[32];
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(o_col + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(rows32 + lane * 256 + ((4 * c + i / 8) ^ (lane & 7)) * 16) =
                make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                           pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
        }
        __syncwarp();
      }
      const int extent = seq.extent(slot), l = lane & 15;
#pragma unroll 4
      for (int i = 0; i < 32; i += 2) {
        const int q = i + (lane >> 4), r = quarter * 32 + q;
        if (r >= extent) continue;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < valid) v = *reinterpret_cast<const uint4*>(rows32 + q * 256 + (l ^ (q & 7)) * 16);
        *reinterpret_cast<uint4*>(head_row(a.out, b, head, seq.start(slot) + r) + 8 * l) = v;
      }
      if (own)
        a.lse[(static_cast<long long>(b) * a.heads + head) * a.rows + row] =
            rloc < valid ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kAtTmem);
  }
}

// Row statistics for the backward pass, per (item, head, slot): 128 values of
// lse in log2 units, then 128 of D = sum_d dO O. Rows not in use get lse =
// +inf (their probabilities become 0) and D = 0. Half a warp per row, 16 bytes
// per lane; bound by reading O and dO.
//
// O was rounded to bf16, and dS = P (dP - D) inherits that error of D. Where
// many keys share a row's weight |O| is well below |V| and the error goes
// unseen; over a handful of keys it is the largest of all. Up to kStatKeys keys
// D is therefore summed as sum_j P_j (dO V_j) from the inputs.
// Over 2, 4, 8 and 16 keys of normal inputs dQ is off by 0.24 % of its norm (the
// roundings of dS and dQ), where O's rounding made that 0.35, 0.28, 0.27 and 0.25.
// The whole backward pass of 4 x 24 heads takes 14.7 us with it at 8 keys and 16.9
// at 16 (13.3 and 13.7 without; 25 at 32, where it gains nothing to speak of).
// Those loops want 114 registers, the plain ones 30: where the rows after the text
// are more than that many already, FEW is false and the loops are not compiled in.
template <bool FEW>
__global__ void __launch_bounds__(256) attn_stat_kernel(const AttnTrainArgs a) {
  pdl_trigger();
  pdl_wait();
  const int slot = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
  const Slots seq(a, b);
  const int valid = seq.valid(slot), start = seq.start(slot);
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  float* stat = a.stats + ((static_cast<long long>(b) * a.heads + head) * a.slots + slot) * 256;
  const int keys = seq.len + a.rows - a.n_txt;
  if (FEW && keys <= kStatKeys) {
    const int kv_head = head / (a.heads / a.kv_heads);
    for (int i = 0; i < 8; ++i) {
      const int r = i * 16 + half;
      float lse = INFINITY, d = 0.f;
      if (i * 16 < valid) {  // the same for the whole block
        uint4 q = make_uint4(0, 0, 0, 0), g = q;
        if (r < valid) {
          lse = a.lse[(static_cast<long long>(b) * a.heads + head) * a.rows + start + r] * kLog2e;
          if (lse == -INFINITY) lse = INFINITY;
          q = *reinterpret_cast<const uint4*>(head_row(a.q, b, head, start + r) + 8 * l);
          g = *reinterpret_cast<const uint4*>(head_row(a.dout, b, head, start + r) + 8 * l);
        }
        for (int j = 0; j < keys; j += 8) {
          uint4 k[8], v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int at = j + u < keys ? j + u : keys - 1;
            const int row = at < seq.len ? at : a.n_txt + at - seq.len;
            k[u] = *reinterpret_cast<const uint4*>(head_row(a.k, b, kv_head, row) + 8 * l);
            v[u] = *reinterpret_cast<const uint4*>(head_row(a.v, b, kv_head, row) + 8 * l);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            float s = dot8(q, k[u]);
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            if (j + u < keys) d = fmaf(fast_exp2(fmaf(s, a.scale_log2, -lse)), dot8(g, v[u]), d);
          }
        }
      }
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
      if (l == 0) {
        stat[r] = lse;
        stat[128 + r] = d;
      }
    }
    return;
  }
#pragma unroll 4
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + half;
    float d = 0.f;
    if (r < valid) {
      const uint4 o = *reinterpret_cast<const uint4*>(head_row(a.out, b, head, start + r) + 8 * l);
      const uint4 g = *reinterpret_cast<const uint4*>(head_row(a.dout, b, head, start + r) + 8 * l);
      d = dot8(o, g);
    }
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    if (l == 0) {
      float lse = INFINITY;
      if (r < valid) {
        lse = a.lse[(static_cast<long long>(b) * a.heads + head) * a.rows + start + r] * kLog2e;
        if (lse == -INFINITY) lse = INFINITY;
      }
      stat[r] = lse;
      stat[128 + r] = d;
    }
  }
}

// Backward. The first blocks make dK and dV, one key slot of one key head
// each, going through the query slots of every query head that shares it; the
// rest make dQ, one query slot of one head each, going through the key slots.
// Recomputing the scores in both costs 7 products instead of 5, but no sum
// is shared between blocks: no atomics, no fp32 copy of dQ in memory, and the
// same bits every run. Both kinds are one grid, so that the second fills the
// SMs that the first leaves at its end.
//
// Roles (576 threads): warp 0 TMA, warp 1 MMA issue, warps 2..17 elementwise,
// four per TMEM lane quarter, each with 32 of the tile's columns. P and dS are
// packed to bf16 over the scores they came from (each warp over its own
// columns) and fed to the next product from tensor memory.
//
// dK/dV block: lanes are keys, columns queries. S^T = K Q^T and dP^T = V dO^T;
// dV += P^T dO, dK += dS^T Q. Tensor memory: S^T | dP^T | dV | dK, 128 columns
// each. While the warps make P_j the tensor core runs dK_{j-1} and dP_j;
// while they make dS_j it runs dV_j and S_{j+1}.
// dQ block: lanes are queries, columns keys. S = Q K^T (two buffers), dP = dO V^T,
// dQ += dS K.
//
// Measured (24 heads, 4608 rows): 700 us in short bursts, 930 TFLOP/s counted as 5 products; 840 in a long loop, at
// the power cap. A dK/dV step takes 3050 clocks for 2048 of tensor work: it waits about 700 for P, whose 16384
// exponentials alone take 1024 (half of them as polynomials on the FMA pipe: 1.5 % faster in all, not kept). A dQ step
// takes 2230 for 1536. CTA pairs, each CTA with half of every streamed operand, were no faster (785 against 764 then).
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_train_bwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                          const AttnTrainArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sm_x = smem;                    // resident: K (Q in a dQ block)
  uint8_t* sm_y = smem + kAtTile;          // resident: V (dO)
  uint8_t* sm_s = smem + kBwdRingS;        // [3]: Q (K)
  uint8_t* sm_t = smem + kBwdRingT;        // [2]: dO (V)
  float* sm_stat = reinterpret_cast<float*>(smem + kBwdStat);  // [2][lse 128 | D 128], dK/dV blocks
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBwdBar);
  uint64_t* x_full = bars + 0;
  uint64_t* s_in = bars + 1;       // [3] first streamed tile
  uint64_t* s_empty = bars + 4;    // [3]
  uint64_t* t_in = bars + 7;       // [2] second streamed tile and the statistics
  uint64_t* t_empty = bars + 9;    // [2] the tile
  uint64_t* stat_empty = bars + 11;  // [2] the statistics, read until dS has been made
  uint64_t* s_full = bars + 13;    // [2] scores ready (dK/dV blocks use the first)
  uint64_t* dp_full = bars + 15;
  uint64_t* p_ready = bars + 16;   // P in tensor memory (dK/dV blocks)
  uint64_t* ds_ready = bars + 17;
  uint64_t* done = bars + 18;
  uint64_t* scrub = bars + 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int kv_blocks = a.slots * a.kv_heads * a.batch;
  const bool is_kv = static_cast<int>(blockIdx.x) < kv_blocks;
  const int group = a.heads / a.kv_heads;
  const int bid = is_kv ? blockIdx.x : blockIdx.x - kv_blocks;
  const int slot = bid % a.slots;
  const int bh = bid / a.slots;
  const int n_heads = is_kv ? a.kv_heads : a.heads;
  const int head = bh % n_heads;  // key head (query head in a dQ block)
  const int b = bh / n_heads;

  if (warp == 0 && lane == 0) {
    mbar_init(x_full, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&s_in[s], 1);
      mbar_init(&s_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&t_in[s], 1);
      mbar_init(&t_empty[s], 1);
      mbar_init(&stat_empty[s], kBwdWarps);
      mbar_init(&s_full[s], 1);
    }
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kBwdWarps);
    mbar_init(ds_ready, kBwdWarps);
    mbar_init(done, 1);
    mbar_init(scrub, 1);
    fence_barrier_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    tma_prefetch_desc(&map_do);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kAtTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_trigger();
  pdl_wait();  // inputs, statistics and outputs are touched only after the previous kernel completes

  const Slots seq(a, b);
  const int valid = seq.valid(slot), start = seq.start(slot);
  const int used = seq.used();
  const int n = valid > 0 ? (is_kv ? used * group : used) : 0;

  if (warp == 0) {
    if (n > 0) {
      StageLog slog, tlog;
      if (lane == 0) {
        mbar_arrive_expect_tx(x_full, 2 * kAtTile);
        tile_load(sm_x, is_kv ? &map_k : &map_q, x_full, start, head, b);
        tile_load(sm_y, is_kv ? &map_v : &map_do, x_full, start, head, b);
      }
      const CUtensorMap* ms = is_kv ? &map_q : &map_k;
      const CUtensorMap* mt = is_kv ? &map_do : &map_v;
      int scrubs = 0;
      int ss = 0;            // stage and phase of the first ring
      uint32_t sp = 0;
      for (int j = 0; j < n; ++j) {
        const int st = j & 1;
        const uint32_t tp = (j >> 1) & 1;
        const int h = is_kv ? head * group + j / used : head / group;
        const int from = seq.used_slot(is_kv ? j % used : j);
        const int row = seq.start(from);
        const bool ragged = seq.ragged(from);
        const uint32_t second = kAtTile + (is_kv ? kStatBytes : 0);
        uint64_t* sb = ragged ? scrub : &s_in[ss];
        uint64_t* tb = ragged ? scrub : &t_in[st];
        if (!mbar_wait_warp(&s_empty[ss], sp ^ 1, 0x411)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(sb, kAtTile + (ragged ? second : 0));
          if (!ragged) slog.armed(ss, sp);
          tile_load(sm_s + ss * kAtTile, ms, sb, row, h, b);
        }
        __syncwarp();
        if (!mbar_wait_warp(&t_empty[st], tp ^ 1, 0x41d)) break;
        if (lane == 0) {
          if (!ragged) {
            mbar_arrive_expect_tx(tb, second);
            tlog.armed(st, tp);
          }
          tile_load(sm_t + st * kAtTile, mt, tb, row, h, b);
        }
        __syncwarp();
        if (is_kv) {
          if (!mbar_wait_warp(&stat_empty[st], tp ^ 1, 0x41e)) break;
          if (lane == 0)
            bulk_load(sm_stat + st * 256, a.stats + ((static_cast<long long>(b) * a.heads + h) * a.slots + from) * 256,
                      kStatBytes, tb);
          __syncwarp();
        }
        if (ragged) {  // rows not in use are summed over by the products: zeros
          if (!mbar_wait_warp(scrub, scrubs & 1, 0x41b)) break;
          ++scrubs;
          scrub_rows(sm_s + ss * kAtTile, seq.valid(from), lane);
          scrub_rows(sm_t + st * kAtTile, seq.valid(from), lane);
          if (lane == 0) {
            mbar_arrive(&s_in[ss]);
            mbar_arrive(&t_in[st]);
            slog.armed(ss, sp);  // the logs hold each stage's latest phase
            tlog.armed(st, tp);
          }
          __syncwarp();
        }
        if (++ss == 3) { ss = 0; sp ^= 1; }
      }
      // no TMA write may land in shared memory after the CTA exits
      if (lane == 0 && mbar_wait(x_full, 0, 0x419)) {
        slog.drain(s_in, 3, 0x419);
        tlog.drain(t_in, 2, 0x419);
      }
    }
  } else if (warp == 1) {
    if (n > 0) {  // the whole warp, see umma_bf16_warp
      bool ok = mbar_wait_warp(x_full, 0, 0x412);
      int si = 0, su = 0;  // first ring: stage of the next tile to wait for, of the step's tile
      uint32_t sp = 0;
      auto wait_s = [&]() -> const uint8_t* {  // the next first tile, or null
        if (!mbar_wait_warp(&s_in[si], sp, 0x413)) return nullptr;
        tc_fence_after();
        const uint8_t* tile = sm_s + si * kAtTile;
        if (++si == 3) { si = 0; sp ^= 1; }
        return tile;
      };
      auto wait_t = [&](int j) {
        const bool r = mbar_wait_warp(&t_in[j & 1], (j >> 1) & 1, 0x413);
        if (r) tc_fence_after();
        return r;
      };
      const uint32_t t_s = tmem_base;
      const uint8_t* tile = nullptr;
      ok = ok && (tile = wait_s()) != nullptr;
      if (ok) {
        mma_along(t_s, sm_x, tile);
        umma_commit_warp(&s_full[0]);
        ok = wait_t(0);
      }
      if (is_kv) {
        const uint32_t t_dp = tmem_base + 128, t_dv = tmem_base + 256, t_dk = tmem_base + 384;
        if (ok) {
          mma_along(t_dp, sm_y, sm_t);
          umma_commit_warp(dp_full);
        }
        for (int j = 0; ok && j < n; ++j) {
          const int st = j & 1, nx = (j + 1) & 1;
          if (!mbar_wait_warp(p_ready, j & 1, 0x414)) break;
          tc_fence_after();
          mma_across_bwd(t_dv, t_s, sm_t + st * kAtTile, j > 0);
          umma_commit_warp(&t_empty[st]);
          if (j + 1 < n) {
            if (!(tile = wait_s())) break;
            mma_along(t_s, sm_x, tile);
            umma_commit_warp(&s_full[0]);
          }
          if (!mbar_wait_warp(ds_ready, j & 1, 0x415)) break;
          tc_fence_after();
          mma_across_bwd(t_dk, t_dp, sm_s + su * kAtTile, j > 0);
          umma_commit_warp(&s_empty[su]);
          if (++su == 3) su = 0;
          if (j + 1 < n) {
            if (!wait_t(j + 1)) break;
            mma_along(t_dp, sm_y, sm_t + nx * kAtTile);
            umma_commit_warp(dp_full);
          }
        }
      } else {
        const uint32_t t_dp = tmem_base + 256, t_dq = tmem_base + 384;
        if (ok) {
          mma_along(t_dp, sm_y, sm_t);
          umma_commit_warp(dp_full);
          umma_commit_warp(&t_empty[0]);
        }
        for (int j = 0; ok && j < n; ++j) {
          const int nx = (j + 1) & 1;
          if (j + 1 < n) {  // the buffer of S_{j-1}, which dS_{j-1} was made from
            if (!(tile = wait_s())) break;
            mma_along(t_s + nx * 128, sm_x, tile);
            umma_commit_warp(&s_full[nx]);
          }
          if (!mbar_wait_warp(ds_ready, j & 1, 0x416)) break;
          tc_fence_after();
          mma_across_bwd(t_dq, t_dp, sm_s + su * kAtTile, j > 0);
          umma_commit_warp(&s_empty[su]);
          if (++su == 3) su = 0;
          if (j + 1 < n) {
            if (!wait_t(j + 1)) break;
            mma_along(t_dp, sm_y, sm_t + nx * kAtTile);
            umma_commit_warp(dp_full);
            umma_commit_warp(&t_empty[nx]);
          }
        }
      }
      // every MMA issued here has completed before the results are read and TMEM is freed
      umma_commit_warp(done);
      mbar_wait_warp(done, 0, 0x41a);
    }
  } else {
    constexpr int kC = kBwdCols;
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;  // which kC of the columns
    const int rloc = quarter * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + part * kC;
    const float sl2 = a.scale_log2;
    bool ok = true;
    float p[kC], d[kC];
    uint32_t pk[kC / 2];
    auto hand_over = [&](uint32_t col, uint64_t* bar) {  // the packed values, to the MMA warp
      tmem_st16(col, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    if (is_kv) {
      for (int j = 0; j < n; ++j) {
        // the statistics come with the second streamed tile
        const float4* lse = reinterpret_cast<const float4*>(sm_stat + (j & 1) * 256 + part * kC);
        const float4* dd = lse + 32;
        if (!mbar_wait_warp(&t_in[j & 1], (j >> 1) & 1, 0x417) || !mbar_wait_warp(&s_full[0], j & 1, 0x417)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(lane_base, p);
#pragma unroll
        for (int i = 0; i < kC; i += 4) {
          const float4 m = lse[i >> 2];
          ffma2(p[i], p[i + 1], p[i], p[i + 1], sl2, sl2, -m.x, -m.y);
          ffma2(p[i + 2], p[i + 3], p[i + 2], p[i + 3], sl2, sl2, -m.z, -m.w);
#pragma unroll
          for (int c = i; c < i + 4; ++c) p[c] = fast_exp2(p[c]);
          pk[i >> 1] = pack_bf16(p[i], p[i + 1]);
          pk[(i >> 1) + 1] = pack_bf16(p[i + 2], p[i + 3]);
        }
        hand_over(lane_base, p_ready);
        if (!mbar_wait_warp(dp_full, j & 1, 0x418)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(lane_base + 128, d);
#pragma unroll
        for (int i = 0; i < kC; i += 4) {
          const float4 m = dd[i >> 2];
          pk[i >> 1] = pack_bf16(p[i] * (d[i] - m.x), p[i + 1] * (d[i + 1] - m.y));
          pk[(i >> 1) + 1] = pack_bf16(p[i + 2] * (d[i + 2] - m.z), p[i + 3] * (d[i + 3] - m.w));
        }
        hand_over(lane_base + 128, ds_ready);
        if (lane == 0) mbar_arrive(&stat_empty[j & 1]);
      }
    } else {
      const float* stat = a.stats + ((static_cast<long long>(b) * a.heads + head) * a.slots + slot) * 256;
      const float lse = stat[rloc], dd = stat[128 + rloc];
      for (int j = 0; j < n; ++j) {
        if (!mbar_wait_warp(&s_full[j & 1], (j >> 1) & 1, 0x417)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(lane_base + (j & 1) * 128, p);
#pragma unroll
        for (int i = 0; i < kC; i += 2) {
          ffma2(p[i], p[i + 1], p[i], p[i + 1], sl2, sl2, -lse, -lse);
          p[i] = fast_exp2(p[i]);
          p[i + 1] = fast_exp2(p[i + 1]);
        }
        const int lim = seq.valid(seq.used_slot(j)) - part * kC;
        if (lim < kC) {
#pragma unroll
          for (int i = 0; i < kC; ++i) p[i] = i < lim ? p[i] : 0.f;
        }
        if (!mbar_wait_warp(dp_full, j & 1, 0x418)) { ok = false; break; }
        tc_fence_after();
        tmem_ld32(lane_base + 256, d);
#pragma unroll
        for (int i = 0; i < kC; i += 2) pk[i >> 1] = pack_bf16(p[i] * (d[i] - dd), p[i + 1] * (d[i + 1] - dd));
        hand_over(lane_base + 256, ds_ready);
      }
    }
    // The results leave through shared memory (the first ring: everything
    // loaded into it has been read), so that a warp writes whole rows of 256
    // bytes. From each lane's own row, 16 bytes in each of 32 rows at a time,
    // this took 7000 clocks of a dK/dV block's 117000, and takes 2500.
    const bool finished = ok && (n == 0 || mbar_wait_warp(done, 0, 0x41c));
    if (finished && n > 0) {
      tc_fence_after();
      auto stage = [&](int at, uint32_t col, float f) {
        tmem_ld32(lane_base + col, d);
        uint8_t* row = sm_s + at * kAtTile + rloc * 256;
#pragma unroll
        for (int i = 0; i < kC; i += 8)
          *reinterpret_cast<uint4*>(row + (((part * kC + i) / 8) ^ (rloc & 7)) * 16) =
              make_uint4(pack_bf16(d[i] * f, d[i + 1] * f), pack_bf16(d[i + 2] * f, d[i + 3] * f),
                         pack_bf16(d[i + 4] * f, d[i + 5] * f), pack_bf16(d[i + 6] * f, d[i + 7] * f));
      };
      if (is_kv) {
        stage(0, 256, 1.0f);
        stage(1, 384, a.scale);
      } else {
        stage(0, 384, a.scale);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kBwdWarps) : "memory");  // the elementwise warps, finished or not
    if (finished) {
      const int extent = seq.extent(slot);
      const int l = lane & 15;  // 16 bytes of a row
      auto write = [&](const HeadsView& view, int at) {
#pragma unroll
        for (int i = 0; i < 128 / kBwdWarps; i += 2) {
          const int r = (warp - 2) * (128 / kBwdWarps) + i + (lane >> 4);
          if (r >= extent) continue;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < valid) v = *reinterpret_cast<const uint4*>(sm_s + at * kAtTile + r * 256 + (l ^ (r & 7)) * 16);
          *reinterpret_cast<uint4*>(head_row(view, b, head, start + r) + 8 * l) = v;
        }
      };
      if (is_kv) {
        write(a.dv, 0);
        write(a.dk, 1);
      } else {
        write(a.dq, 0);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kAtTmem);
  }
}

// ------------------------------------------------------------------ host

static int make_heads_map(CUtensorMap* map, const HeadsView& v, int rows, int heads, int batch) {
  return make_map_4d(map, v.data, kHeadDim, rows, heads, batch, static_cast<uint64_t>(v.row_stride) * 2,
                     static_cast<uint64_t>(v.head_stride) * 2, static_cast<uint64_t>(v.batch_stride) * 2, 64, 128);
}

template <typename K>
static int opt_in_smem(K kernel, int bytes, bool* configured) {
  const int dev = current_device();
  if (dev < 0) return -1;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return -1;
    configured[dev] = true;
  }
  return 0;
}

int launch_attention_train(const AttnTrainArgs& a, cudaStream_t s) {
  static bool configured[kMaxDevices] = {};
  if (opt_in_smem(attn_train_fwd_kernel, kFwdSmem, configured)) return -1;
  CUtensorMap mq, mk, mv;
  if (make_heads_map(&mq, a.q, a.rows, a.heads, a.batch) || make_heads_map(&mk, a.k, a.rows, a.kv_heads, a.batch) ||
      make_heads_map(&mv, a.v, a.rows, a.kv_heads, a.batch))
    return -2;
  const cudaError_t e = launch_kernel(attn_train_fwd_kernel, dim3((a.slots + 1) / 2, a.heads, a.batch),
                                      dim3(kAtThreads), kFwdSmem, s, 1, mq, mk, mv, a);
  note_launch();
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

int launch_attention_backward(const AttnTrainArgs& a, cudaStream_t s) {
  static bool configured[kMaxDevices] = {};
  if (opt_in_smem(attn_train_bwd_kernel, kBwdSmem, configured)) return -1;
  CUtensorMap mq, mk, mv, md;
  if (make_heads_map(&mq, a.q, a.rows, a.heads, a.batch) || make_heads_map(&mk, a.k, a.rows, a.kv_heads, a.batch) ||
      make_heads_map(&mv, a.v, a.rows, a.kv_heads, a.batch) || make_heads_map(&md, a.dout, a.rows, a.heads, a.batch))
    return -2;
  auto stat = a.rows - a.n_txt <= kStatKeys ? attn_stat_kernel<true> : attn_stat_kernel<false>;
  cudaError_t e = launch_kernel(stat, dim3(a.slots, a.heads, a.batch), dim3(256), 0, s, 1, a);
  note_launch();
  if (e == cudaSuccess) {
    const int blocks = a.slots * (a.kv_heads + a.heads) * a.batch;
    e = launch_kernel(attn_train_bwd_kernel, dim3(blocks), dim3(kBwdThreads), kBwdSmem, s, 1, mq, mk, mv, md, a);
    note_launch();
  }
  return (e == cudaSuccess && cudaPeekAtLastError() == cudaSuccess) ? 0 : -1;
}

}  // namespace klein
