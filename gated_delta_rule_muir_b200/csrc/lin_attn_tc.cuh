// Linear attention with one decay per head: the tensor-core pass for bf16 inputs.
// lin_attn.cuh has the formulas and what a pass is.
//
// One CTA per (pass, sequence, head, segment) walks its segment in chunks of 128
// tokens. Per chunk, with operand tiles a, b, c of 128 tokens and S the state
// before the chunk (products on tcgen05, accumulators in TMEM):
//
//   scores = a b^T                        128 x 128
//   y1 = (scores o decay mask) c          the weights rounded once to bf16
//   y2 = a S                              S rounded once to bf16 as an operand
//   dS = (b weight)^T c                   fp32-exact: see below
//   out_i = y1_i + o_scale lambda^(..) y2_i,   S <- lambda^128 S + dS
//
// The decay of a head is one number, so it enters y2 as a row factor in fp32 after
// the product and the scores as a factor per element before their one rounding.
// Only dS has a factor inside a product whose result must stay fp32: each row of b
// times its weight (an fp32 number) is cut into three bf16 parts that sum to it
// exactly, and three products are accumulated. S itself lives in registers in
// fp32, is updated by fp32 adds (never accumulated in TMEM from chunk to chunk),
// and only its operand copy is rounded. So y has one bf16 rounding of each weight
// and of the state, and the final state is fp32.
//
// Six products of 128 x 128 x 128 per chunk are 3072 tensor cycles of the about
// 5700 that 128 KB of operands and output take at this GPU's copy bandwidth with
// one CTA per SM: the pass is bound by memory when the tiles of the next chunk
// arrive while this one computes. Shared memory decides that: 32 KB per tile, a
// ring of five slots for a, b, c (the next chunk's a and b land during this
// chunk, its c when this chunk's a has been used), one tile for S, and one for the
// parts of b: the first part is written over b once the scores are done, the
// second beside it, the third over the first: 224 KB.
//
// Roles (512 threads): warp 0 issues TMA copies, warp 1 the MMAs; warps 4..7 (one
// token row per thread) mask the scores and write outputs; warps 8..15 cut b and
// keep the state (one row, 64 columns per thread). Hand-offs are mbarriers with
// bounded waits:
//   full[s], empty[s]   slot s holds a tile / its last reader is done
//   scores    scores in TMEM               (MMA -> mask, cut)
//   weights   masked scores in TMEM        (mask -> MMA)
//   y         y1 and y2 in TMEM            (MMA -> mask)
//   y_free    y1 and y2 read               (mask -> MMA)
//   cut12, cut3   parts 1 and 2 / 3 of b in shared memory (cut -> MMA)
//   used12    parts 1 and 2 used           (MMA -> cut)
//   ds        dS in TMEM                   (MMA -> state)
//   s_ready   S for the next chunk in shared memory (state -> MMA)
#pragma once

#include "lin_attn.cuh"
#include "tma.cuh"

namespace muir {

constexpr int kLtChunk = 128;
constexpr int kLtThreads = 512;
constexpr uint32_t kLtTile = 32768, kLtBox = 16384;  // 128 rows x 128 columns bf16: two boxes of 64 columns
// slots of the ring: with outputs five (beside S and the part tile), without six
template <bool OUT> constexpr int kLtSlots = OUT ? 5 : 6;
constexpr uint32_t kLtSmem = 7 * kLtTile + 1024;

constexpr int kLinMaxPasses = 3;
struct LinTcArgs {
  CUtensorMap a[kLinMaxPasses], b[kLinMaxPasses], c[kLinMaxPasses];
  LinPass p[kLinMaxPasses];
};

// One box of 64 channels x 128 tokens of one sequence; tokens past T read as zeros.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tmap, int x, int y, int z, uint64_t* bar) {
  MUIR_SMEM_GUARD(dst, 16384u);
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A whole warp's wait: every lane gets the same answer, so that the aligned
// instructions after it are reached by all lanes or by none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

// A operand in TMEM (row = lane, two bf16 per column).
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// 16 columns (32-bit words) of this thread's lane; completes before return.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 bf16 (8 words) to global memory: one 32-byte store where p is 32-byte
// aligned, else two of 16 bytes.
__device__ __forceinline__ void stg_bf16x16(__nv_bfloat16* p, const uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// One (pass, sequence, head, segment) of a launch.
struct LinUnit {
  int b, h, bh, seg;
  int64_t t0, valid;  // first token, valid tokens
  int chunks;
  float c2;           // log2 lambda
};
__device__ __forceinline__ LinUnit lin_unit(const LinPass& p) {
  LinUnit u;
  u.seg = (int)(blockIdx.x % p.nseg);
  u.bh = (int)(blockIdx.x / p.nseg);
  u.b = u.bh / p.H;
  u.h = u.bh % p.H;
  u.t0 = (int64_t)u.seg * p.seglen;
  u.valid = lin_seg_tokens(p, lin_length(p, u.b), u.seg);
  u.chunks = (int)((u.valid + kLtChunk - 1) / kLtChunk);
  u.c2 = lin_log2(p.log_decay, u.h);
  return u;
}

template <bool OUT>
__global__ void __launch_bounds__(kLtThreads, 1) lin_tc_kernel(const __grid_constant__ LinTcArgs args) {
  extern __shared__ __align__(1024) uint8_t lt_sm[];
  constexpr int SLOTS = kLtSlots<OUT>;
  constexpr int TILES = OUT ? 3 : 2;  // per chunk: a, b, c or b, c
  __shared__ uint64_t full[SLOTS], empty[SLOTS], b_scores, b_weights, b_y, b_yfree, b_cut12, b_cut3, b_used12, b_ds, b_sready;
  __shared__ uint32_t tslot;
  const int pi = blockIdx.y;
  const LinPass& p = args.p[pi];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const LinUnit u = lin_unit(p);
  const uint32_t base = (smem_u32(lt_sm) + 1023u) & ~1023u;
  const uint32_t s_tile = base + 5u * kLtTile, x_tile = base + 6u * kLtTile;  // without outputs s_tile is slot 5
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&b_scores, 1);
    mbar_init(&b_weights, 4);
    mbar_init(&b_y, 1);
    mbar_init(&b_yfree, 4);
    mbar_init(&b_cut12, 8);
    mbar_init(&b_cut3, 8);
    mbar_init(&b_used12, 1);
    mbar_init(&b_ds, 1);
    mbar_init(&b_sready, 8);
  }
  if (warp == 0) tmem_alloc(&tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;
  const uint32_t t_scores = tmem, t_y1 = tmem + 128, t_y2 = tmem + 256, t_ds = tmem + 384;
  // chunk n of the walk: its place in the segment
  auto chunk_at = [&](int n) { return p.reverse ? u.chunks - 1 - n : n; };

  if (warp == 0) {
    // ---- TMA: tiles in the order they are needed, a(n) b(n) c(n) a(n+1) .. --------
    if (lane == 0) {
      const int abytes = p.da > 64 ? 32768 : 16384, cbytes = p.dc > 64 ? 32768 : 16384;
      bool ok = true;
      int m = 0;
      for (int n = 0; n < u.chunks && ok; ++n) {
        const int t = (int)(u.t0 + (int64_t)chunk_at(n) * kLtChunk);
        for (int k = OUT ? 0 : 1; k < 3 && ok; ++k, ++m) {
          const int s = m % SLOTS, turn = m / SLOTS;
          if (turn > 0) ok = mbar_wait(&empty[s], (uint32_t)(turn - 1) & 1u);
          if (!ok) break;
          const CUtensorMap* map = k == 0 ? &args.a[pi] : k == 1 ? &args.b[pi] : &args.c[pi];
          const int d = k == 2 ? p.dc : p.da;
          const uint32_t dst = base + (uint32_t)s * kLtTile;
          mbar_expect_tx(&full[s], (uint32_t)(k == 2 ? cbytes : abytes));
          tma_load_3d(dst, map, u.h * d, t, u.b, &full[s]);
          if (d > 64) tma_load_3d(dst + kLtBox, map, u.h * d + 64, t, u.b, &full[s]);
        }
      }
      // no copy is in flight when the CTA ends, even after a wait that ran out
      for (int s = 0; s < SLOTS; ++s)
        if (m > s) mbar_wait(&full[s], (uint32_t)((m - 1 - s) / SLOTS) & 1u);
    }
  } else if (warp == 1) {
    // ---- MMA ------------------------------------------------------------------------
    if (lane == 0) {
      bool ok = true;
      const int ka = p.da / 16;
      const uint32_t id_scores = idesc_bf16(128, 128, 0, 0), id_y = idesc_bf16(128, p.dc, 0, 1),
                     id_ds = idesc_bf16(128, p.dc, 1, 1);
      auto part = [&](uint32_t bt, uint32_t ct, bool accum) {  // dS (+)= part^T c
        for (int j = 0; j < 8; ++j)
          mma_bf16(t_ds, sdesc_sw128(bt + (uint32_t)j * 2048u, kLtBox, 1024u), sdesc_sw128(ct + (uint32_t)j * 2048u, kLtBox, 1024u),
                   id_ds, accum || j > 0 ? 1u : 0u);
      };
      for (int n = 0; n < u.chunks && ok; ++n) {
        const uint32_t ph = (uint32_t)n & 1u;
        const int m = n * TILES;
        const int sa = m % SLOTS, sb = (m + TILES - 2) % SLOTS, sc = (m + TILES - 1) % SLOTS;
        const uint32_t at = base + (uint32_t)sa * kLtTile, bt = base + (uint32_t)sb * kLtTile, ct = base + (uint32_t)sc * kLtTile;
        if (OUT) {
          ok = mbar_wait(&full[sa], (uint32_t)(m / SLOTS) & 1u) && mbar_wait(&full[sb], (uint32_t)((m + 1) / SLOTS) & 1u);
          if (ok && n > 0) ok = mbar_wait(&b_y, ph ^ 1u);  // the last weights have been used
          if (!ok) break;
          tc_fence_after();
          for (int j = 0; j < ka; ++j) {
            const uint32_t o = (uint32_t)(j >> 2) * kLtBox + (uint32_t)(j & 3) * 32u;
            mma_bf16(t_scores, sdesc_sw128(at + o, 16u, 1024u), sdesc_sw128(bt + o, 16u, 1024u), id_scores, j > 0 ? 1u : 0u);
          }
          mma_commit(&b_scores);
          ok = mbar_wait(&b_sready, ph);
          if (ok && n > 0) ok = mbar_wait(&b_yfree, ph ^ 1u);
          if (!ok) break;
          tc_fence_after();
          for (int j = 0; j < ka; ++j) {
            const uint32_t o = (uint32_t)(j >> 2) * kLtBox + (uint32_t)(j & 3) * 32u;
            mma_bf16(t_y2, sdesc_sw128(at + o, 16u, 1024u), sdesc_sw128(s_tile + (uint32_t)j * 2048u, kLtBox, 1024u), id_y,
                     j > 0 ? 1u : 0u);
          }
          mma_commit(&empty[sa]);
        }
        ok = mbar_wait(&full[sc], (uint32_t)((m + TILES - 1) / SLOTS) & 1u) && mbar_wait(&b_cut12, ph);
        if (!ok) break;
        tc_fence_after();
        part(bt, ct, false);
        part(x_tile, ct, true);
        mma_commit(&b_used12);
        if (OUT) {
          ok = mbar_wait(&b_weights, ph);
          if (!ok) break;
          tc_fence_after();
          for (int j = 0; j < 8; ++j)
            mma_bf16_ta(t_y1, t_scores + (uint32_t)j * 8u, sdesc_sw128(ct + (uint32_t)j * 2048u, kLtBox, 1024u), id_y,
                        j > 0 ? 1u : 0u);
          mma_commit(&b_y);
        }
        ok = mbar_wait(&b_cut3, ph);
        if (!ok) break;
        tc_fence_after();
        part(bt, ct, true);
        mma_commit(&empty[sb]);
        mma_commit(&empty[sc]);
        mma_commit(&b_ds);
      }
      // every issued product has completed when the CTA ends: each chunk's last commit
      // is waited for here, or after a wait that ran out one more commit is
      if (ok) {
        if (u.chunks > 0) mbar_wait(&b_ds, (uint32_t)(u.chunks - 1) & 1u);
      } else {
        mma_commit(&b_ds);
        mbar_wait_for(&b_ds, 0u, 1000000ull);
        mbar_wait_for(&b_ds, 1u, 1000000ull);
      }
    }
  } else if (OUT && warp >= 4 && warp < 8) {
    // ---- mask and outputs: thread = token row i of the chunk ----------------------------
    const int w = warp & 3, i = w * 32 + lane;
    const uint32_t row = tmem_lane_base(warp);
    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.out) + (((int64_t)u.b * p.T + u.t0) * p.H + u.h) * p.dc;
    const int64_t pitch = (int64_t)p.H * p.dc;
    {  // padded tokens of this segment: zeros
      const int64_t end = (u.t0 + p.seglen < p.T ? p.seglen : p.T - u.t0);
      const int pieces = p.dc / 8;
      for (int64_t x = u.valid * pieces + i; x < end * pieces; x += 128)
        *reinterpret_cast<uint4*>(out + (x / pieces) * pitch + (x % pieces) * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
    // lambda^gap = (row factor of a block of 32 columns) (column factor in the block),
    // both at most 1 for blocks off the diagonal
    float cf[32];
#pragma unroll
    for (int s = 0; s < 32; ++s) cf[s] = exp2f(u.c2 * (float)(p.reverse ? s : 31 - s));
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const uint32_t ph = (uint32_t)n & 1u;
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      ok = warp_wait(&b_scores, ph);
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t wd[16];
        const bool none = p.reverse ? k < w : k > w;
        if (none) {  // whole warp: masked block
#pragma unroll
          for (int q = 0; q < 16; ++q) wd[q] = 0u;
        } else {
          float v[32];
          tmem_ld32(t_scores + row + (uint32_t)(32 * k), v);
          if (k == w) {
#pragma unroll
            for (int s = 0; s < 32; ++s) {
              const int gap = p.reverse ? s - lane : lane - s;
              // dropped, not multiplied by zero: a masked score may be anything
              v[s] = gap >= 0 && 32 * k + s < L ? v[s] * (p.p_scale * exp2f(u.c2 * (float)gap)) : 0.f;
            }
          } else {
            const float rf = p.p_scale * exp2f(u.c2 * (float)(p.reverse ? 32 * k - i : i - 32 * k - 31));
#pragma unroll
            for (int s = 0; s < 32; ++s) v[s] = 32 * k + s < L ? v[s] * (rf * cf[s]) : 0.f;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) wd[q] = bf16x2(v[2 * q], v[2 * q + 1]);
        }
        // columns 16 k .. of the scores have been read: block k's weights go there
        tmem_st16(t_scores + row + (uint32_t)(16 * k), wd);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_weights);
      ok = warp_wait(&b_y, ph);
      if (!ok) break;
      tc_fence_after();
      const float rw = p.o_scale * exp2f(u.c2 * (float)(p.reverse ? (i < L ? L - 1 - i : 0) : i + 1));
#pragma unroll 1
      for (int c = 0; c < p.dc; c += 32) {
        float y1[32], y2[32];
        tmem_ld32(t_y1 + row + (uint32_t)c, y1);
        tmem_ld32(t_y2 + row + (uint32_t)c, y2);
        if (c + 32 >= p.dc) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive1(&b_yfree);
        }
        if (i < L) {
          __nv_bfloat16* d = out + (r0 + i) * pitch + c;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              o[q] = bf16x2(fmaf(rw, y2[16 * hf + 2 * q], y1[16 * hf + 2 * q]),
                            fmaf(rw, y2[16 * hf + 2 * q + 1], y1[16 * hf + 2 * q + 1]));
            stg_bf16x16(d + 16 * hf, o);
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ---- cut b, keep the state ------------------------------------------------------------
    const int half = (warp - 8) >> 2;            // columns 64 half .. of b's tile and of S
    const int r = (warp & 3) * 32 + lane;        // token row of b's tile; row of S
    const uint32_t row = tmem_lane_base(warp);
    const int nstate = p.da * p.dc;
    const bool mine = r < p.da && 64 * half < p.dc;       // has a row of S
    const int scols = p.dc - 64 * half < 64 ? p.dc - 64 * half : 64;
    float S[64];
    {
      const float* src = nullptr;
      bool tr = false;
      if constexpr (OUT) {
        if (p.seg) { src = p.seg + ((int64_t)u.bh * p.nseg + u.seg) * nstate; tr = p.seg_t; }
        else if (p.init) { src = p.init + (int64_t)u.bh * nstate; tr = p.init_t; }
      }
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        S[j] = 0.f;
        if (src && mine && j < scols)
          S[j] = tr ? __ldg(src + (int64_t)(64 * half + j) * p.da + r) : __ldg(src + (int64_t)r * p.dc + 64 * half + j);
      }
    }
    auto put_state = [&]() {  // S's operand copy: row r, columns 64 half ..
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (mine && 8 * c < scols) {
          uint4 v;
          v.x = bf16x2(S[8 * c], S[8 * c + 1]);
          v.y = bf16x2(S[8 * c + 2], S[8 * c + 3]);
          v.z = bf16x2(S[8 * c + 4], S[8 * c + 5]);
          v.w = bf16x2(S[8 * c + 6], S[8 * c + 7]);
          sts128(s_tile + (uint32_t)half * kLtBox + (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7)) << 4), v);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_sready);
    };
    if constexpr (OUT) put_state();
    const int bcols = p.da - 64 * half < 64 ? p.da - 64 * half : 64;  // of b's tile, at most 0: none
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const uint32_t ph = (uint32_t)n & 1u;
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      const int m = n * TILES + TILES - 2;
      const int sb = m % SLOTS, sc = (m + 1) % SLOTS;
      const uint32_t line = base + (uint32_t)sb * kLtTile + (uint32_t)half * kLtBox + (uint32_t)r * 128u;
      const uint32_t xline = x_tile + (uint32_t)half * kLtBox + (uint32_t)r * 128u;
      const float wt = r < L ? p.u_scale * exp2f(u.c2 * (float)(p.reverse ? r + 1 : L - 1 - r)) : 0.f;
      ok = warp_wait(&full[sb], (uint32_t)(m / SLOTS) & 1u) && warp_wait(&full[sc], (uint32_t)((m + 1) / SLOTS) & 1u);
      if (OUT && ok) ok = warp_wait(&b_scores, ph);  // b itself has been used
      if (!ok) break;
      uint32_t third[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t at = (uint32_t)((c ^ (r & 7)) << 4);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (8 * c < bcols) v = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(line + at));
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t p1[4], p2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          // rows past the last token become zeros whatever they hold
          float f0 = r < L ? __uint_as_float(in[q] << 16) * wt : 0.f;
          float f1 = r < L ? __uint_as_float(in[q] & 0xFFFF0000u) * wt : 0.f;
          p1[q] = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
          f0 -= __uint_as_float(__float_as_uint(f0) & 0xFFFF0000u);
          f1 -= __uint_as_float(__float_as_uint(f1) & 0xFFFF0000u);
          p2[q] = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
          f0 -= __uint_as_float(__float_as_uint(f0) & 0xFFFF0000u);
          f1 -= __uint_as_float(__float_as_uint(f1) & 0xFFFF0000u);
          third[4 * c + q] = __byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x7632);
        }
        if (8 * c < bcols) {
          sts128(line + at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
          sts128(xline + at, make_uint4(p2[0], p2[1], p2[2], p2[3]));
        }
      }
      if (r >= L) {  // c's rows past the last token: zero times anything must stay zero
        const uint32_t cline = base + (uint32_t)sc * kLtTile + (uint32_t)half * kLtBox + (uint32_t)r * 128u;
#pragma unroll
        for (int c = 0; c < 8; ++c) sts128(cline + (uint32_t)(c << 4), make_uint4(0u, 0u, 0u, 0u));
      }
      fence_async_smem();
      tc_fence_before();  // this thread's reads of the last dS precede the next
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_cut12);
      ok = warp_wait(&b_used12, ph);
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (8 * c < bcols)
          sts128(line + (uint32_t)((c ^ (r & 7)) << 4),
                 make_uint4(third[4 * c], third[4 * c + 1], third[4 * c + 2], third[4 * c + 3]));
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_cut3);
      ok = warp_wait(&b_ds, ph);
      if (!ok) break;
      tc_fence_after();
      const float wl = exp2f(u.c2 * (float)L);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (64 * half + 32 * hf < p.dc) {  // whole warps
          float d[32];
          tmem_ld32(t_ds + row + (uint32_t)(64 * half + 32 * hf), d);
#pragma unroll
          for (int j = 0; j < 32; ++j) S[32 * hf + j] = fmaf(wl, S[32 * hf + j], d[j]);
        }
      }
      if (OUT && n + 1 < u.chunks) put_state();
    }
    float* dst = nullptr;
    if constexpr (!OUT) dst = p.seg + ((int64_t)u.bh * p.nseg + u.seg) * nstate;
    else if (p.fin && p.nseg == 1) dst = p.fin + (int64_t)u.bh * nstate;
    if (dst && mine) {
      dst += (int64_t)r * p.dc + 64 * half;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (8 * c < scols) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = S[8 * c + j];
          stg256(dst + 8 * c, v);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace muir
