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
// Roles (768 threads): warp 0 issues TMA copies, warp 1 the MMAs; warps 4..7 (one
// token row per thread) mask the scores and write outputs; warps 8..15 cut b (half
// a token row per thread); warps 16..23 keep the state (one row, 64 columns per
// thread). The products are issued y1(n), parts 1 and 2 (n), scores(n+1), part 3
// (n), y2(n+1), so that the scores fill the wait for the third part and the
// masking, cutting and outputs of one chunk run under the products of another.
// The block is launched with 80 registers per thread; the warpgroups trade them
// (64 + 96 + 2 x 64 + 2 x 96 = 6 x 80). Hand-offs are mbarriers with bounded
// waits:
//   full[s], empty[s]   slot s holds a tile / its last reader is done
//   scores    scores in TMEM               (MMA -> mask, cut)
//   weights   masked scores in TMEM        (mask -> MMA)
//   y         y1 and y2 in TMEM            (MMA -> mask)
//   y_free    y1 and y2 read               (mask -> MMA)
//   cut12, cut3   parts 1 and 2 / 3 of b in shared memory (cut -> MMA)
//   used12    parts 1 and 2 used           (MMA -> cut)
//   ds        dS in TMEM                   (MMA -> state, cut)
//   ds_free   dS read                      (state -> MMA)
//   s_ready   S for the next chunk in shared memory (state -> MMA)
#pragma once

#include "lin_attn.cuh"
#include "tma.cuh"

namespace muir {

constexpr int kLtChunk = 128;
constexpr int kLtThreads = 768;
constexpr uint32_t kLtTile = 32768, kLtBox = 16384;  // 128 rows x 128 columns bf16: two boxes of 64 columns
constexpr int kLtSlots = 5;
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

// One MMA with the accumulate flag known at compile time. The issuing thread must
// not be slower than the tensor core (64 cycles for 128 x 128 x 16): with unrolled
// steps, constant offsets added to one descriptor and constant flags a step takes
// 65 cycles; with flags and step counts from registers it took 180 to 270.
template <bool ACC>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// The same with the A operand in TMEM (row = lane, two bf16 per column).
template <bool ACC>
__device__ __forceinline__ void mma_step_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}

// Step j of 16 channels of a K-major tile / of 16 rows of an MN-major one, in
// descriptor units of 16 bytes.
__host__ __device__ constexpr uint64_t lt_kstep(int j) { return (uint64_t)(((j >> 2) * kLtBox + (j & 3) * 32u) >> 4); }
__host__ __device__ constexpr uint64_t lt_mnstep(int j) { return (uint64_t)((j * 2048u) >> 4); }

template <int STEPS, bool ACC, bool A_MN, bool B_MN>
__device__ __forceinline__ void lt_product(uint32_t d_tmem, uint32_t at, uint32_t bt, uint32_t idesc) {
  const uint64_t a = sdesc_sw128(at, A_MN ? kLtBox : 16u, 1024u), b = sdesc_sw128(bt, B_MN ? kLtBox : 16u, 1024u);
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const uint64_t aj = a + (A_MN ? lt_mnstep(j) : lt_kstep(j)), bj = b + (B_MN ? lt_mnstep(j) : lt_kstep(j));
    if (ACC || j > 0) mma_step<true>(d_tmem, aj, bj, idesc);
    else mma_step<false>(d_tmem, aj, bj, idesc);
  }
}
// over 32, 64 or 128 channels
template <bool B_MN>
__device__ __forceinline__ void lt_product_k(int channels, uint32_t d_tmem, uint32_t at, uint32_t bt, uint32_t idesc) {
  if (channels == 128) lt_product<8, false, false, B_MN>(d_tmem, at, bt, idesc);
  else if (channels == 64) lt_product<4, false, false, B_MN>(d_tmem, at, bt, idesc);
  else lt_product<2, false, false, B_MN>(d_tmem, at, bt, idesc);
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

// 32 columns from each of two places of this thread's lane: both loads, one wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, uint32_t tb, float (&a)[32], float (&b)[32]) {
  uint32_t r[32], s[32];
  auto issue = [](uint32_t t, uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]),
          "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]),
          "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(t)
        : "memory");
  };
  issue(ta, r);
  issue(tb, s);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) {  // after the wait: the registers are not valid before it
    asm volatile("" : "+r"(r[i]), "+r"(s[i]));
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(s[i]);
  }
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

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

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

template <bool OUT, int PARTS>
__global__ void __launch_bounds__(kLtThreads, 1) lin_tc_kernel(const __grid_constant__ LinTcArgs args) {
  extern __shared__ __align__(1024) uint8_t lt_sm[];
  constexpr int SLOTS = kLtSlots;
  constexpr int TILES = OUT ? 3 : 2;  // per chunk: a, b, c or b, c
  __shared__ uint64_t full[SLOTS], empty[SLOTS], b_scores, b_weights, b_y2, b_y, b_yfree, b_cut12, b_cut3, b_used12, b_ds, b_dsfree, b_sready;
  __shared__ uint32_t tslot;
  __shared__ float pw[kLtChunk];              // lambda^0 ..
  __shared__ __align__(16) float pcol[32];    // column factors inside a block of 32 (see the mask)
  const int pi = blockIdx.y;
  const LinPass p = args.p[pi];  // by value: the waits between uses would reload what a reference names
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const LinUnit u = lin_unit(p);
  const uint32_t base = (smem_u32(lt_sm) + 1023u) & ~1023u;
  // beside the ring: the second parts' tile, and S's or (without outputs) a second one
  const uint32_t x_tile = base + 5u * kLtTile, s_tile = base + 6u * kLtTile;
  auto x_of = [&](int n) { return OUT ? x_tile : x_tile + (uint32_t)(n & 1) * kLtTile; };
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&b_scores, 1);
    mbar_init(&b_weights, 4);
    mbar_init(&b_y2, 1);
    mbar_init(&b_y, 1);
    mbar_init(&b_yfree, 4);
    mbar_init(&b_cut12, 8);
    mbar_init(&b_cut3, 8);
    mbar_init(&b_used12, 1);
    mbar_init(&b_ds, 1);
    mbar_init(&b_dsfree, 8);
    mbar_init(&b_sready, 8);
  }
  if (warp == 0) tmem_alloc(&tslot, 512);
  if (tid < kLtChunk) pw[tid] = exp2f(u.c2 * (float)tid);
  if (tid < 32) pcol[tid] = exp2f(u.c2 * (float)(p.reverse ? tid : 31 - tid));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;
  const uint32_t t_scores = tmem, t_y1 = tmem + 128, t_y2 = tmem + 256, t_ds = tmem + 384;
  // chunk n of the walk: its place in the segment
  auto chunk_at = [&](int n) { return p.reverse ? u.chunks - 1 - n : n; };

  if (warp < 4) {
    regs_dec<64>();
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
    // The warp stays converged and one elected lane issues: slots, step counts and
    // waits' results are the same in every lane and known to be (a vote, a warp
    // reduction), so that the descriptors are formed in uniform registers. Issued
    // from inside a one-lane branch, each product took three to four times as long.
    const bool leader = elect_one();
    const int chunks = (int)__reduce_max_sync(0xffffffffu, (unsigned)u.chunks);
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const uint32_t m_scores = tm, m_y1 = tm + 128, m_y2 = tm + 256, m_ds = tm + 384;
    bool ok = true;
    const uint32_t id_scores = idesc_bf16(128, 128, 0, 0), id_y = idesc_bf16(128, p.dc, 0, 1),
                   id_ds = idesc_bf16(128, p.dc, 1, 1);
    auto slot = [&](int m) { return base + (uint32_t)(m % SLOTS) * kLtTile; };
    auto landed = [&](int m) { return warp_wait(&full[m % SLOTS], (uint32_t)(m / SLOTS) & 1u); };
    auto scores = [&](int n) {  // a b^T of chunk n; its TMEM columns hold chunk n - 1's weights until y1 is done
      const int m = n * TILES;
      if (!landed(m) || !landed(m + 1) || (n > 0 && !warp_wait(&b_y, (uint32_t)(n - 1) & 1u))) return false;
      tc_fence_after();
      if (leader) {
        lt_product_k<false>(p.da, m_scores, slot(m), slot(m + 1), id_scores);
        mma_commit(&b_scores);
      }
      __syncwarp();
      return true;
    };
    if (OUT && chunks > 0) ok = scores(0);
    for (int n = 0; n < chunks && ok; ++n) {
      const uint32_t ph = (uint32_t)n & 1u;
      const int ma = n * TILES, mb = ma + TILES - 2, mc = ma + TILES - 1;
      const uint32_t at = slot(ma), bt = slot(mb), ct = slot(mc);
      // c's tile: landed, and its rows past the last token cleared by the cutters
      ok = landed(mc) && warp_wait(&b_cut12, ph) && (n == 0 || warp_wait(&b_dsfree, ph ^ 1u));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        lt_product<8, false, true, true>(m_ds, bt, ct, id_ds);
        lt_product<8, true, true, true>(m_ds, x_of(n), ct, id_ds);
        mma_commit(PARTS == 2 ? &b_ds : &b_used12);
      }
      __syncwarp();
      if (OUT) {
        ok = warp_wait(&b_sready, ph) && (n == 0 || warp_wait(&b_yfree, ph ^ 1u));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          lt_product_k<true>(p.da, m_y2, at, s_tile, id_y);
          mma_commit(&b_y2);
          mma_commit(&empty[ma % SLOTS]);
        }
        __syncwarp();
        ok = warp_wait(&b_weights, ph);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t cd = sdesc_sw128(ct, kLtBox, 1024u);
          mma_step_ta<false>(m_y1, m_scores, cd, id_y);
#pragma unroll
          for (int j = 1; j < 8; ++j) mma_step_ta<true>(m_y1, m_scores + (uint32_t)j * 8u, cd + lt_mnstep(j), id_y);
          mma_commit(&b_y);
          if (PARTS == 2) {
            mma_commit(&empty[mb % SLOTS]);
            mma_commit(&empty[mc % SLOTS]);
          }
        }
        __syncwarp();
        if (n + 1 < chunks) ok = scores(n + 1);
      }
      if (PARTS == 3) {
        ok = ok && warp_wait(&b_cut3, ph);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          lt_product<8, true, true, true>(m_ds, bt, ct, id_ds);
          mma_commit(&b_ds);
          mma_commit(&empty[mb % SLOTS]);
          mma_commit(&empty[mc % SLOTS]);
        }
        __syncwarp();
      }
    }
    // every issued product has completed when the CTA ends: the last chunk's commits
    // are waited for here, or after a wait that ran out one more commit is
    if (ok) {
      if (chunks > 0) {
        warp_wait(&b_ds, (uint32_t)(chunks - 1) & 1u);
        if (OUT) warp_wait(&b_y, (uint32_t)(chunks - 1) & 1u);
      }
    } else {
      if (leader) mma_commit(&b_ds);
      __syncwarp();
      mbar_wait_for(&b_ds, 0u, 1000000ull);
      mbar_wait_for(&b_ds, 1u, 1000000ull);
    }
    }
  } else if (warp < 8) {
    // ---- mask and outputs: thread = token row i of the chunk ----------------------------
    regs_inc<96>();
    if constexpr (OUT) {
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
            const int last = L - 32 * k;  // columns from here on are past the last token
#pragma unroll
            for (int s = 0; s < 32; ++s) {
              const int gap = p.reverse ? s - lane : lane - s;
              const float f = v[s] * (p.p_scale * pw[gap & 31]);
              // dropped, not multiplied by zero: a masked score may be anything
              v[s] = (gap >= 0) & (s < last) ? f : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) wd[q] = bf16x2(v[2 * q], v[2 * q + 1]);
          } else {
            const float rf = p.p_scale * pw[p.reverse ? 32 * k - i : i - 32 * k - 31];
            const float2 rf2 = make_float2(rf, rf);
            if (32 * k + 32 > L) {  // columns past the last token
#pragma unroll
              for (int s = 0; s < 32; ++s) v[s] = 32 * k + s < L ? v[s] : 0.f;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 cf = *reinterpret_cast<const float4*>(&pcol[4 * q]);
              const float2 f = __fmul2_rn(make_float2(v[4 * q], v[4 * q + 1]), __fmul2_rn(make_float2(cf.x, cf.y), rf2));
              const float2 g = __fmul2_rn(make_float2(v[4 * q + 2], v[4 * q + 3]), __fmul2_rn(make_float2(cf.z, cf.w), rf2));
              wd[2 * q] = bf16x2(f.x, f.y);
              wd[2 * q + 1] = bf16x2(g.x, g.y);
            }
          }
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
      const float rw = p.o_scale * (p.reverse ? pw[i < L ? L - 1 - i : 0] : exp2f(u.c2 * (float)(i + 1)));
#pragma unroll 1
      for (int c = 0; c < p.dc; c += 32) {
        float y1[32], y2[32];
        tmem_ld32x2(t_y1 + row + (uint32_t)c, t_y2 + row + (uint32_t)c, y1, y2);
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
            for (int q = 0; q < 8; ++q) {
              const int e = 16 * hf + 2 * q;
              const float2 y = __ffma2_rn(make_float2(rw, rw), make_float2(y2[e], y2[e + 1]), make_float2(y1[e], y1[e + 1]));
              o[q] = bf16x2(y.x, y.y);
            }
            stg_bf16x16(d + 16 * hf, o);
          }
        }
      }
    }
    }
  } else if (warp < 16) {
    // ---- cut b: thread = half a token row ---------------------------------------------------
    regs_dec<64>();
    const int half = (warp - 8) >> 2;      // columns 64 half ..
    const int r = (warp & 3) * 32 + lane;  // token row
    const int bcols = p.da - 64 * half < 64 ? p.da - 64 * half : 64;  // at most 0: none
    const uint32_t place = (uint32_t)half * kLtBox + (uint32_t)r * 128u;
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const uint32_t ph = (uint32_t)n & 1u;
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      const int m = n * TILES + TILES - 2;
      const int sb = m % SLOTS, sc = (m + 1) % SLOTS;
      const uint32_t line = base + (uint32_t)sb * kLtTile + place;
      const uint32_t xline = x_of(n) + place;
      const float wt = r < L ? p.u_scale * exp2f(u.c2 * (float)(p.reverse ? r + 1 : L - 1 - r)) : 0.f;
      ok = warp_wait(&full[sb], (uint32_t)(m / SLOTS) & 1u) && warp_wait(&full[sc], (uint32_t)((m + 1) / SLOTS) & 1u);
      if (OUT) {
        ok = ok && warp_wait(&b_scores, ph);  // b itself has been used, and the last second parts
        if (PARTS == 2 && n > 0) ok = ok && warp_wait(&b_ds, ph ^ 1u);
      }
      if (!ok) break;
      uint32_t x[32];  // the half row, then its third parts
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(line + (uint32_t)((c ^ (r & 7)) << 4)));
        x[4 * c] = v.x;
        x[4 * c + 1] = v.y;
        x[4 * c + 2] = v.z;
        x[4 * c + 3] = v.w;
      }
      if (r >= L) {  // rows past the last token count as zeros, whatever they hold
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t p1[4], p2[4];
        const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t in = x[4 * c + q];
          float2 f = __fmul2_rn(make_float2(__uint_as_float(in << 16), __uint_as_float(in & 0xFFFF0000u)), make_float2(wt, wt));
          if (PARTS == 2) {
            p1[q] = bf16x2(f.x, f.y);
            f = __ffma2_rn(make_float2(__uint_as_float(p1[q] << 16), __uint_as_float(p1[q] & 0xFFFF0000u)), minus, f);
            p2[q] = bf16x2(f.x, f.y);
          } else {
            auto upper = [&]() {
              return make_float2(__uint_as_float(__float_as_uint(f.x) & 0xFFFF0000u),
                                 __uint_as_float(__float_as_uint(f.y) & 0xFFFF0000u));
            };
            auto pack = [&]() { return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632); };
            p1[q] = pack();
            f = __ffma2_rn(upper(), minus, f);
            p2[q] = pack();
            f = __ffma2_rn(upper(), minus, f);
            x[4 * c + q] = pack();
          }
        }
        if (8 * c < bcols) {
          const uint32_t at = (uint32_t)((c ^ (r & 7)) << 4);
          sts128(line + at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
          sts128(xline + at, make_uint4(p2[0], p2[1], p2[2], p2[3]));
        }
      }
      if (r >= L) {  // c's rows past the last token: zero times anything must stay zero
        const uint32_t cline = base + (uint32_t)sc * kLtTile + place;
#pragma unroll
        for (int c = 0; c < 8; ++c) sts128(cline + (uint32_t)(c << 4), make_uint4(0u, 0u, 0u, 0u));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_cut12);
      if (PARTS == 3) {
        ok = warp_wait(&b_used12, ph);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (8 * c < bcols)
            sts128(line + (uint32_t)((c ^ (r & 7)) << 4), make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&b_cut3);
      }
    }
  } else {
    // ---- the state: thread = row r, columns 64 half .. -----------------------------------------
    regs_inc<96>();
    const int half = (warp - 16) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t row = tmem_lane_base(warp);
    const int nstate = p.da * p.dc;
    const bool mine = r < p.da && 64 * half < p.dc;
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
    auto put_state = [&]() {  // S's operand copy
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
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      const LinDecay wl = lin_decay(u.c2, L);
      ok = warp_wait(&b_ds, (uint32_t)n & 1u);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (64 * half + 32 * q < p.dc) {  // whole warps
          float d[32];
          tmem_ld32(t_ds + row + (uint32_t)(64 * half + 32 * q), d);
          const float2 g = make_float2(wl.g, wl.g), e = make_float2(wl.e, wl.e);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float* s2 = S + 32 * q + j;
            const float2 old = make_float2(s2[0], s2[1]);
            const float2 now = __ffma2_rn(g, old, __ffma2_rn(e, old, make_float2(d[j], d[j + 1])));
            s2[0] = now.x;
            s2[1] = now.y;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_dsfree);
      if (OUT && n + 1 < u.chunks) {
        ok = warp_wait(&b_y2, (uint32_t)n & 1u);  // the last copy has been used
        if (!ok) break;
        put_state();
      }
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
