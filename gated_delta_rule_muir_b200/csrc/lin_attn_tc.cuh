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
// and of the state, and the final state is fp32. These two are what a bf16 operand costs
// (error of y 0.0020 to 0.0022 of its size, of the gradients 0.0023, where the output's own
// rounding is 0.0017); second parts of both would be two more products a chunk, and 32 KB
// more of shared memory for the state's than there are. fp32 operands avoid both.
//
// An outputs' launch that keeps no final state (one of several segments: the final
// state comes from the segments' own) feeds S only to y, through its bf16 operand copy;
// there b is cut into two parts, rounded to nearest: off by 2^-18 of a product in the
// mean and 1.5 x 2^-15 at most, a 256th of what the operand copy of S loses. It takes
// three packed bf16 operations for two elements; with three parts there too, one sequence
// of 32768 tokens, 16 heads of 128, takes 222 us forward against 196 and 640 backward
// against 558. Segment states, which are carried over whole sequences, are made of three
// parts always (of two, with the same operands: backward 579 us against 593 in long runs).
//
// Bound: per chunk 128 KB of operands and output, about 5700 cycles at this GPU's
// copy bandwidth with one CTA per SM; five products of 512 tensor cycles (six with
// three parts); and shared memory, about 4600 cycles of its 128 bytes a cycle: the
// products read 2300 cycles' worth (a 128 x 128 x 16 step with both operands in shared
// memory takes all of it), copies in and out 1000, cutting 770, S and the outputs 500.
// Spills at 72 registers: 44 bytes a thread with two parts, 148 with three, 4 without outputs.
// Measured, one sequence of 32768 tokens, 16 heads of 128: outputs 124 us (83 at the
// copy bandwidth), the segments' own states 71 (42). With nearly all work on elements
// left out of a timing copy the outputs took 105 us, and no single role's work moved
// them by more than 10: what is left is the traffic and the hand-offs, not one stage.
// Slower were: masking in unrolled blocks of 32 columns (237 us for both launches
// against 220: such code runs at the pace of instruction fetches), outputs stored a
// row per thread, tiles asked into L2 two chunks ahead, y2 issued before the parts.
//
// Shared memory, 7 tiles of 32 KB: a ring of four for b, a, c (b first: it is cut
// ahead of everything else and its slot is free again as soon as it has been cut and
// multiplied), two for the parts, one for S. Third parts of 128 channels
// go over b itself. Without
// outputs: the ring for b, c, first parts over b, two tiles for second parts (even
// and odd chunks) and one for third parts, which are multiplied first.
//
// Roles (896 threads): warp 0 issues TMA copies, warp 1 the MMAs; warps 4..11 mask
// the scores (one token row, every other 16 columns per thread); warps 12..19 cut b
// (half a token row per thread); warps 20..27 keep the state and write outputs (one
// row, 64 columns per thread). The products are issued parts(n), y2(n), y1(n), scores(n+1):
// the parts and y2 run while the scores are masked. The block is launched with 72
// registers per thread; the warpgroups trade them (40 + 2 x 56 + 2 x 64 + 2 x 112 =
// 7 x 72). Without outputs warps 4..19 cut (a quarter row per thread) and dS has two
// buffers in TMEM. Hand-offs are mbarriers with bounded waits:
//   full[s], empty[s]   slot s holds a tile / its readers are done (one commit and the
//                       cutting warps, or for c the warps that write outputs over it)
//   scores    scores in TMEM               (MMA -> mask, cut)
//   weights   masked scores in TMEM        (mask -> MMA)
//   y2, y     y2 / y1 and y2 in TMEM       (MMA -> state)
//   y_free    y1 and y2 read               (state -> MMA)
//   cut       the parts in shared memory   (cut -> MMA)
//   used3     third parts used             (MMA -> cut; without outputs)
//   ds, ds_free   dS in TMEM / read        (MMA -> state, cut / state -> MMA)
//   s_ready   S for the next chunk in shared memory (state -> MMA)
#pragma once

#include "lin_attn.cuh"
#include "tma.cuh"

namespace muir {

constexpr int kLtChunk = 128;
constexpr int kLtThreads = 896;
constexpr uint32_t kLtTile = 32768, kLtBox = 16384;  // 128 rows x 128 columns bf16: two boxes of 64 columns
constexpr int kLtSlots = 4;
constexpr uint32_t kLtSmem = 7 * kLtTile + 1024;

struct LinTcArgs {
  CUtensorMap a[kLinMaxPasses], b[kLinMaxPasses], c[kLinMaxPasses];  // boxes of 64 channels x 128 tokens
  CUtensorMap o[kLinMaxPasses];  // outputs, 64 x 32; unused for 32 channels
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

// One box from shared memory to global memory, in this thread's bulk-async group;
// tokens past T are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tmap, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
// Until this thread's committed bulk copies have read their source.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits of this kernel. Bounded like mbar_wait, with as little code in line as will
// do (there are some twenty of them, and the roles run at the pace of instruction
// fetches): the first try decides nearly always, and the time is only looked at
// every 256 tries after that.
__device__ __forceinline__ bool is_over(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !is_over(bar, parity); ++it) {
    if ((it & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) { flag_timeout(); return false; }
    }
  }
  return true;
}
// A whole warp's wait: every lane gets the same answer, so that the aligned
// instructions after it are reached by all lanes or by none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, lane_wait(bar, parity)) != 0;
}

// One MMA with the accumulate flag known at compile time. The issuing thread must
// not be slower than the tensor core (64 cycles for 128 x 128 x 16): with unrolled
// steps, constant offsets added to one descriptor and constant flags a step takes
// 65 cycles; with flags and step counts from registers it took 180 to 270.
// A descriptor is its low word; the high one (stride of 8-row groups 1024 bytes,
// version, 128-byte swizzle) is the same for every tile here.
constexpr uint32_t kLtDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t lt_desc(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }

template <bool ACC>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %4};\n\t"
      "mov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "n"(kLtDescHi), "n"(ACC ? 1 : 0)
      : "memory");
}
// The same with the A operand in TMEM (row = lane, two bf16 per column).
template <bool ACC>
__device__ __forceinline__ void mma_step_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "n"(kLtDescHi), "n"(ACC ? 1 : 0)
      : "memory");
}

// Step j of 16 channels of a K-major tile / of 16 rows of an MN-major one, in
// descriptor units of 16 bytes.
__host__ __device__ constexpr uint32_t lt_kstep(int j) { return ((j >> 2) * kLtBox + (j & 3) * 32u) >> 4; }
__host__ __device__ constexpr uint32_t lt_mnstep(int j) { return (j * 2048u) >> 4; }

template <int STEPS, bool ACC, bool A_MN, bool B_MN>
__device__ __forceinline__ void lt_product(uint32_t d_tmem, uint32_t at, uint32_t bt, uint32_t idesc) {
  const uint32_t a = lt_desc(at, A_MN ? kLtBox : 16u), b = lt_desc(bt, B_MN ? kLtBox : 16u);
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const uint32_t aj = a + (A_MN ? lt_mnstep(j) : lt_kstep(j)), bj = b + (B_MN ? lt_mnstep(j) : lt_kstep(j));
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

// 8 columns (32-bit words) of this thread's lane; completes before return.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
      : "memory");
}

// 16 columns from each of two places of this thread's lane: both loads, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&a)[16], float (&b)[16]) {
  uint32_t r[16], s[16];
  auto issue = [](uint32_t t, uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
        : "r"(t)
        : "memory");
  };
  issue(ta, r);
  issue(tb, s);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {  // uses come after the wait: the registers are not valid before it
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
  static_assert(OUT || PARTS == 3, "segment states are exact");
  extern __shared__ __align__(1024) uint8_t lt_sm[];
  constexpr int SLOTS = kLtSlots;
  constexpr int TILES = OUT ? 3 : 2;  // per chunk: a, b, c or b, c
  constexpr int CUTTERS = OUT ? 8 : 16;  // warps that cut b: without outputs the mask's warps too
  // dS in one TMEM buffer, or in two in turn where the other accumulators leave room
  auto ds_buf = [](int n) { return OUT ? 0 : n & 1; };
  auto ds_phase = [](int n) { return (uint32_t)(OUT ? n : n >> 1) & 1u; };
  __shared__ uint64_t full[SLOTS], empty[SLOTS], b_scores, b_weights, b_y2, b_y, b_yfree, b_cut, b_used3, b_ds[2], b_dsfree[2], b_sready;
  __shared__ uint32_t tslot;
  __shared__ float pw[kLtChunk];              // lambda^0 ..
  __shared__ __align__(16) float pcol[16];    // column factors of 16 columns (see the mask)
  const int pi = blockIdx.y;
  const LinPass p = args.p[pi];  // by value: the waits between uses would reload what a reference names
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid >= 64 && tid < 68) {  // the descriptors, ahead of their first use
    const int i = tid - 64;
    if (i < 2 || OUT) {
      if (i != 3 || p.dc >= 64) tma_prefetch_desc(i == 0 ? &args.b[pi] : i == 1 ? &args.c[pi] : i == 2 ? &args.a[pi] : &args.o[pi]);
    }
  }
  const LinUnit u = lin_unit(p);
  const uint32_t base = (smem_u32(lt_sm) + 1023u) & ~1023u;
  // the parts of chunk n's b, given b's own tile
  const uint32_t spare = base + (uint32_t)SLOTS * kLtTile, s_tile = spare + 2u * kLtTile;
  auto part1 = [&](int n, uint32_t bt) { return OUT ? spare : bt; };
  auto part2 = [&](int n, uint32_t bt) { return spare + (OUT ? 1u : (uint32_t)(n & 1)) * kLtTile; };
  // third parts of 128 channels go over b, after the scores; of 64 they have room beside the first
  constexpr bool thirds = PARTS == 3;
  const bool over_b = OUT && thirds && p.da > 64;
  auto part3 = [&](int n, uint32_t bt) { return !OUT ? spare + 2u * kLtTile : over_b ? bt : spare + kLtBox; };
  // chunk n of the walk: its place in the segment
  auto chunk_at = [&](int n) { return p.reverse ? u.chunks - 1 - n : n; };
  // tile m of the walk into its slot, in the order b(0) a(0) c(0) b(1) ..
  const int all_tiles = u.chunks * TILES;
  auto load_tile = [&](int m) {
    const int s = m % SLOTS, n = m / TILES, k = m % TILES;
    const CUtensorMap* map = k == 0 ? &args.b[pi] : k == TILES - 1 ? &args.c[pi] : &args.a[pi];
    const int d = k == TILES - 1 ? p.dc : p.da, t = (int)(u.t0 + (int64_t)chunk_at(n) * kLtChunk);
    const uint32_t dst = base + (uint32_t)s * kLtTile;
    mbar_expect_tx(&full[s], d > 64 ? 2u * kLtBox : kLtBox);
    tma_load_3d(dst, map, u.h * d, t, u.b, &full[s]);
    if (d > 64) tma_load_3d(dst + kLtBox, map, u.h * d + 64, t, u.b, &full[s]);
  };
  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1 + CUTTERS);
    }
    mbar_init(&b_scores, 1);
    mbar_init(&b_weights, 8);
    mbar_init(&b_y2, 1);
    mbar_init(&b_y, 1);
    mbar_init(&b_yfree, 8);
    mbar_init(&b_cut, CUTTERS);
    mbar_init(&b_used3, 1);
    mbar_init(&b_ds[0], 1);
    mbar_init(&b_ds[1], 1);
    mbar_init(&b_dsfree[0], 8);
    mbar_init(&b_dsfree[1], 8);
    mbar_init(&b_sready, 8);
    fence_async_smem();
    // the first tiles are on their way while the rest of the CTA sets up
#pragma unroll 1
    for (int m = 0; m < SLOTS && m < all_tiles; ++m) load_tile(m);
  }
  if (warp == 1) tmem_alloc(&tslot, 512);
  if (tid < kLtChunk) pw[tid] = exp2f(u.c2 * (float)tid);
  if (tid < 16) pcol[tid] = exp2f(u.c2 * (float)(p.reverse ? tid : 15 - tid));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tslot;
  const uint32_t t_scores = tmem, t_y1 = tmem + 128, t_y2 = tmem + 256;
  auto t_ds = [&](int n) { return tmem + 384u - 128u * (uint32_t)ds_buf(n); };

  if (warp < 4) {
    regs_dec<40>();
    if (warp == 0) {
      // ---- TMA: the remaining tiles, each as its slot comes free ------------------------
      if (lane == 0) {
        bool ok = true;
        int m = SLOTS < all_tiles ? SLOTS : all_tiles;
        for (; m < all_tiles; ++m) {
          ok = lane_wait(&empty[m % SLOTS], (uint32_t)(m / SLOTS - 1) & 1u);
          if (!ok) break;
          load_tile(m);
        }
        // no copy is in flight when the CTA ends, even after a wait that ran out
        for (int s = 0; s < SLOTS; ++s)
          if (m > s) mbar_wait(&full[s], (uint32_t)((m - 1 - s) / SLOTS) & 1u);
      }
    } else if (warp == 1) {
      // ---- MMA: one elected lane -----------------------------------------------------
      const int chunks = (int)__reduce_max_sync(0xffffffffu, (unsigned)u.chunks);  // known to be the same in all lanes
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
      if (elect_one()) {
        const uint32_t m_scores = tm, m_y1 = tm + 128, m_y2 = tm + 256;
        const uint32_t id_scores = idesc_bf16(128, 128, 0, 0), id_y = idesc_bf16(128, p.dc, 0, 1),
                       id_ds = idesc_bf16(128, p.dc, 1, 1);
        bool ok = true;
        auto slot = [&](int m) { return base + (uint32_t)(m % SLOTS) * kLtTile; };
        auto landed = [&](int m) { return lane_wait(&full[m % SLOTS], (uint32_t)(m / SLOTS) & 1u); };
        auto scores = [&](int n) {  // a b^T of chunk n; its TMEM columns hold chunk n - 1's weights until y1 is done
          const int m = n * TILES;
          if (!landed(m) || !landed(m + 1) || (n > 0 && !lane_wait(&b_y, (uint32_t)(n - 1) & 1u))) return false;
          tc_fence_after();
          lt_product_k<false>(p.da, m_scores, slot(m + 1), slot(m), id_scores);
          mma_commit(&b_scores);
          if (!over_b) mma_commit(&empty[m % SLOTS]);
          return true;
        };
        if (OUT && chunks > 0) ok = scores(0);
        for (int n = 0; n < chunks && ok; ++n) {
          const uint32_t ph = (uint32_t)n & 1u;
          const int mb = n * TILES, ma = mb + 1, mc = mb + TILES - 1;
          const uint32_t bt = slot(mb), ct = slot(mc), m_ds = tm + 384u - 128u * (uint32_t)ds_buf(n);
          // c's tile has landed, and the cutters have cleared its rows past the last token
          ok = landed(mc) && lane_wait(&b_cut, ph) &&
               (n <= ds_buf(1) || lane_wait(&b_dsfree[ds_buf(n)], ds_phase(n) ^ 1u));
          if (!ok) break;
          tc_fence_after();
          if constexpr (thirds) {
            lt_product<8, false, true, true>(m_ds, part3(n, bt), ct, id_ds);
            if (!OUT) mma_commit(&b_used3);
          }
          lt_product<8, thirds, true, true>(m_ds, part2(n, bt), ct, id_ds);
          lt_product<8, true, true, true>(m_ds, part1(n, bt), ct, id_ds);
          mma_commit(&b_ds[ds_buf(n)]);
          if (!OUT || over_b) mma_commit(&empty[mb % SLOTS]);
          if constexpr (!OUT) {
            mma_commit(&empty[mc % SLOTS]);
          } else {
            ok = lane_wait(&b_sready, ph) && (n == 0 || lane_wait(&b_yfree, ph ^ 1u));
            if (!ok) break;
            tc_fence_after();
            lt_product_k<true>(p.da, m_y2, slot(ma), s_tile, id_y);
            mma_commit(&b_y2);
            mma_commit(&empty[ma % SLOTS]);
            ok = lane_wait(&b_weights, ph);
            if (!ok) break;
            tc_fence_after();
            const uint32_t cd = lt_desc(ct, kLtBox);
            mma_step_ta<false>(m_y1, m_scores, cd, id_y);
#pragma unroll
            for (int j = 1; j < 8; ++j) mma_step_ta<true>(m_y1, m_scores + (uint32_t)(16 * j), cd + lt_mnstep(j), id_y);
            mma_commit(&b_y);
            mma_commit(&empty[mc % SLOTS]);
            if (n + 1 < chunks) ok = scores(n + 1);
          }
        }
        // every issued product has completed when the CTA ends: the last chunk's commits
        // are waited for here, or after a wait that ran out one more commit is
        if (ok) {
          if (chunks > 0) {
            lane_wait(&b_ds[ds_buf(chunks - 1)], ds_phase(chunks - 1));
            if (OUT) lane_wait(&b_y, (uint32_t)(chunks - 1) & 1u);
          }
        } else {
          mma_commit(&b_scores);
          mbar_wait_for(&b_scores, 0u, 1000000ull);
          mbar_wait_for(&b_scores, 1u, 1000000ull);
        }
      }
    }
  } else if (OUT && warp < 12) {
    // ---- mask: thread = token row i of the chunk, every other 16 columns -------------------------
    regs_dec<56>();
    const int w = warp & 3, i = w * 32 + lane, c0 = warp < 8 ? 0 : 16;
    const uint32_t row = tmem_lane_base(warp);
    // 16 columns at a time in one short loop (an unrolled body of this size runs at the
    // pace of instruction fetches). lambda^gap = (row factor) (column factor), the
    // column factor at most 1 and the row factor at most lambda^-15, 2^60 for decays
    // above 2^-4; below that, and for scales above 2^60, which would take the row factor
    // out of range, the powers are taken from the table one by one.
    const bool mild = u.c2 > -4.f && fabsf(p.p_scale) <= 0x1p60f;
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const uint32_t ph = (uint32_t)n & 1u;
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      ok = warp_wait(&b_scores, ph);
      if (!ok) break;
      tc_fence_after();
      auto skip = [&](int c) { return p.reverse ? c + 15 < 32 * w : c > 32 * w + 31; };  // nothing counts for the warp's rows
#pragma unroll 1
      for (int c = c0; c < 128; c += 32) {
        // columns lo .. hi - 1 of the 16 count
        const int lo = p.reverse ? i - c : 0, hi = (p.reverse ? L : (i + 1 < L ? i + 1 : L)) - c;
        uint32_t wd[8];
        if (skip(c)) {
#pragma unroll
          for (int q = 0; q < 8; ++q) wd[q] = 0u;
        } else {
          float v[16];
          tmem_ld16(t_scores + row + (uint32_t)c, v);
          const int e = p.reverse ? c - i : i - c - 15;
          if (mild) {
            const float rf = p.p_scale * exp2f(u.c2 * (float)max(e, -15));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 cf = *reinterpret_cast<const float4*>(&pcol[4 * q]);
              const float2 f = __fmul2_rn(make_float2(v[4 * q], v[4 * q + 1]), __fmul2_rn(make_float2(cf.x, cf.y), make_float2(rf, rf)));
              const float2 g = __fmul2_rn(make_float2(v[4 * q + 2], v[4 * q + 3]), __fmul2_rn(make_float2(cf.z, cf.w), make_float2(rf, rf)));
              v[4 * q] = f.x;
              v[4 * q + 1] = f.y;
              v[4 * q + 2] = g.x;
              v[4 * q + 3] = g.y;
            }
          } else {
#pragma unroll
            for (int s = 0; s < 16; ++s) v[s] *= p.p_scale * pw[max(0, p.reverse ? e + s : e + 15 - s)];
          }
          if (__any_sync(0xffffffffu, lo > 0 || hi < 16)) {
            // dropped, not multiplied by zero: what does not count may be anything
#pragma unroll
            for (int s = 0; s < 16; ++s) v[s] = (s >= lo) & (s < hi) ? v[s] : 0.f;
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) wd[q] = bf16x2(v[2 * q], v[2 * q + 1]);
        }
        // over the first half of the scores they come from
        tmem_st8(t_scores + row + (uint32_t)c, wd);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&b_weights);
    }
  } else if (warp < 20) {
    // ---- cut b: thread = half a token row --------------------------------------------------------
    regs_dec<64>();
    constexpr int PIECES = OUT ? 8 : 4;                 // 8-column pieces of the row per thread
    const int q0 = ((warp - (OUT ? 12 : 4)) >> 2) * PIECES;  // first of them
    const int r = (warp & 3) * 32 + lane;  // token row
    const uint32_t place = (uint32_t)(q0 >> 3) * kLtBox + (uint32_t)r * 128u;
    const int k0 = q0 & 7;  // in the box's row
    bool ok = true;
    for (int n = 0; n < u.chunks && ok; ++n) {
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      const int mb = n * TILES, mc = mb + TILES - 1;
      const uint32_t bt = base + (uint32_t)(mb % SLOTS) * kLtTile;
      const uint32_t line = bt + place, l1 = part1(n, bt) + place, l2 = part2(n, bt) + place, l3 = part3(n, bt) + place;
      const float wt = r < L ? p.u_scale * exp2f(u.c2 * (float)(p.reverse ? r + 1 : L - 1 - r)) : 0.f;
      ok = warp_wait(&full[mb % SLOTS], (uint32_t)(mb / SLOTS) & 1u);
      // the tiles of the last parts have been used; before third parts go over b, the scores have been formed
      if (n > 0) ok = ok && warp_wait(OUT ? &b_ds[0] : &b_used3, (uint32_t)(n - 1) & 1u);
      // c only after that: the last parts came behind the scores of their chunk, so the tile
      // before c's in its slot (a's of that chunk) has landed, and a parity names one phase
      if (L < kLtChunk) ok = ok && warp_wait(&full[mc % SLOTS], (uint32_t)(mc / SLOTS) & 1u);
      if (over_b) ok = ok && warp_wait(&b_scores, (uint32_t)n & 1u);
      if (!ok) break;
      // packed bf16, two parts: with the weight as w1 + w2, p1 = b w1 rounded, and
      // p2 = (b w1 - p1) + b w2, the bracket exact, rounded once
      const __nv_bfloat16 w1 = __float2bfloat16_rn(wt), w2 = __float2bfloat16_rn(wt - __bfloat162float(w1));
      const __nv_bfloat162 w11 = __halves2bfloat162(w1, w1), w22 = __halves2bfloat162(w2, w2);
      if (8 * q0 < p.da) {
#pragma unroll 4
        for (int c = k0; c < k0 + PIECES; ++c) {
          const uint32_t at = (uint32_t)((c ^ (r & 7)) << 4);
          uint4 v = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(line + at));
          if (r >= L) v = make_uint4(0u, 0u, 0u, 0u);  // past the last token: zeros, whatever they hold
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          uint32_t p1[4], p2[4], p3[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (PARTS == 3) {  // the upper 16 bits of the fp32 product, of its rest, of the rest of that
              float2 f = __fmul2_rn(make_float2(__uint_as_float(in[q] << 16), __uint_as_float(in[q] & 0xFFFF0000u)),
                                    make_float2(wt, wt));
              auto rest = [&]() {
                const uint32_t hi = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
                f = __ffma2_rn(make_float2(__uint_as_float(__float_as_uint(f.x) & 0xFFFF0000u),
                                           __uint_as_float(__float_as_uint(f.y) & 0xFFFF0000u)),
                               make_float2(-1.f, -1.f), f);
                return hi;
              };
              p1[q] = rest();
              p2[q] = rest();
              p3[q] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
            } else {
              const __nv_bfloat162 bb = *reinterpret_cast<const __nv_bfloat162*>(&in[q]);
              const __nv_bfloat162 h = __hmul2(bb, w11);
              const __nv_bfloat162 l = __hfma2(bb, w22, __hfma2(bb, w11, __hneg2(h)));
              p1[q] = *reinterpret_cast<const uint32_t*>(&h);
              p2[q] = *reinterpret_cast<const uint32_t*>(&l);
            }
          }
          // (columns past da hold other heads' channels: cut as well, rows of dS that nobody reads)
          sts128(l1 + at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
          sts128(l2 + at, make_uint4(p2[0], p2[1], p2[2], p2[3]));
          if constexpr (thirds) sts128(l3 + at, make_uint4(p3[0], p3[1], p3[2], p3[3]));
        }
      }
      if (r >= L) {  // c's rows past the last token: zero times anything must stay zero
        const uint32_t cline = base + (uint32_t)(mc % SLOTS) * kLtTile + place;
        for (int c = k0; c < k0 + PIECES; ++c) sts128(cline + (uint32_t)((c ^ (r & 7)) << 4), make_uint4(0u, 0u, 0u, 0u));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive1(&b_cut);
        for (int m = mb; m < mc; ++m) mbar_arrive1(&empty[m % SLOTS]);
        if (!OUT) mbar_arrive1(&empty[mc % SLOTS]);
      }
    }
  } else {
    // ---- the state and outputs: thread = row r, columns 64 half .. -----------------------------------
    regs_inc<OUT ? 112 : 104>();
    const int half = (warp - 20) >> 2;
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
      for (int j = 0; j < 64; ++j) S[j] = 0.f;
      if (src && mine && tr) {
        src += (int64_t)(64 * half) * p.da + r;
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (j < scols) S[j] = __ldg(src + j * p.da);
      } else if (src && mine) {
        src += (int64_t)r * p.dc + 64 * half;
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          if (j < scols) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(src + j));
            S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
          }
        }
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
    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.out) + (((int64_t)u.b * p.T + u.t0) * p.H + u.h) * p.dc;
    const int64_t pitch = (int64_t)p.H * p.dc;
    if constexpr (OUT) {  // padded tokens of this segment: zeros
      const int64_t end = (u.t0 + p.seglen < p.T ? p.seglen : p.T - u.t0);
      const int pieces = p.dc / 8;
      for (int64_t x = u.valid * pieces + tid - 640; x < end * pieces; x += 256)
        *reinterpret_cast<uint4*>(out + (x / pieces) * pitch + (x % pieces) * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
    // outputs of chunk n: row r, columns 64 half .. They are laid down in c's tile, which
    // y1 has read by then, and copied out by the warp's own TMA store, in whole lines
    // (a token row per thread stored directly takes a pass of the load-store unit per
    // row and instruction: 1700 of the chunk's 7000 cycles). 32 channels are half a
    // box; those go directly.
    const bool boxed = p.dc >= 64;
    auto outputs = [&](int n) {
      const int64_t r0 = (int64_t)chunk_at(n) * kLtChunk;
      const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
      if (!warp_wait(&b_y, (uint32_t)n & 1u)) return false;
      tc_fence_after();
      const float rw = p.o_scale * (p.reverse ? pw[r < L ? L - 1 - r : 0] : exp2f(u.c2 * (float)(r + 1)));
      const float2 rw2 = make_float2(rw, rw);
      const uint32_t stage = base + (uint32_t)((n * TILES + TILES - 1) % SLOTS) * kLtTile + (uint32_t)half * kLtBox + (uint32_t)r * 128u;
#pragma unroll 1
      for (int c = 64 * half; c < 64 * half + 64 && c < p.dc; c += 16) {
        float y1[16], y2[16];
        tmem_ld16x2(t_y1 + row + (uint32_t)c, t_y2 + row + (uint32_t)c, y1, y2);
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 y = __ffma2_rn(rw2, make_float2(y2[2 * q], y2[2 * q + 1]), make_float2(y1[2 * q], y1[2 * q + 1]));
          o[q] = r < L ? bf16x2(y.x, y.y) : 0u;  // padded tokens: zeros
        }
        if (boxed) {
          const uint32_t k = (uint32_t)((c & 63) >> 3);
          sts128(stage + (((k ^ (uint32_t)(r & 7))) << 4), make_uint4(o[0], o[1], o[2], o[3]));
          sts128(stage + ((((k + 1) ^ (uint32_t)(r & 7))) << 4), make_uint4(o[4], o[5], o[6], o[7]));
        } else if (r < L) {
          stg_bf16x16(out + (r0 + r) * pitch + c, o);
        }
      }
      tc_fence_before();
      if (boxed) fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive1(&b_yfree);
        if (boxed && 64 * half < p.dc) {
          tma_store_3d(&args.o[pi], stage, u.h * p.dc + 64 * half, (int)(u.t0 + r0) + r, u.b);
          bulk_commit();
        }
      }
      return true;
    };
    // c's tile of chunk n may be filled again
    auto release_c = [&](int n) {
      if (lane == 0) {
        bulk_wait_read();
        mbar_arrive1(&empty[(n * TILES + TILES - 1) % SLOTS]);
      }
    };
    bool ok = true;
    // step n: S after chunk n - 1, its operand copy for chunk n, the outputs of chunk n - 1
    for (int n = OUT ? 0 : 1; n <= u.chunks && ok; ++n) {
      if (n > 0) {
        const int64_t r0 = (int64_t)chunk_at(n - 1) * kLtChunk;
        const int L = (int)(u.valid - r0 < kLtChunk ? u.valid - r0 : kLtChunk);
        const LinDecay wl = lin_decay(u.c2, L);
        ok = warp_wait(&b_ds[ds_buf(n - 1)], ds_phase(n - 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (64 * half + 16 * q < p.dc) {  // whole warps
            float d[16];
            tmem_ld16(t_ds(n - 1) + row + (uint32_t)(64 * half + 16 * q), d);
            const float2 g = make_float2(wl.g, wl.g), e = make_float2(wl.e, wl.e);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float* s2 = S + 16 * q + j;
              const float2 old = make_float2(s2[0], s2[1]);
              const float2 now = __ffma2_rn(g, old, __ffma2_rn(e, old, make_float2(d[j], d[j + 1])));
              s2[0] = now.x;
              s2[1] = now.y;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&b_dsfree[ds_buf(n - 1)]);
      }
      if constexpr (OUT) {
        if (n < u.chunks) {
          if (n > 0) ok = warp_wait(&b_y2, (uint32_t)(n - 1) & 1u);  // the last copy has been used
          if (!ok) break;
          put_state();
        }
        if (n > 0) {
          ok = outputs(n - 1);
          release_c(n - 1);
        }
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
    if (OUT && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace muir
