// kld_packed_rows.cu -- the statistic and the gradient with packed base rows
// (mathematics: kld_packed_rows.cuh).
//
// Both passes in one launch. A row belongs to one CTA of four warps, or, when
// there are few rows, to a cluster of 2, 4 or 8 of them, each taking a run of
// its 512-column chunks. A warp streams its chunks, two at a
// time, through shared-memory slots of its own with cp.async (every global
// read whole 16-byte vectors in order), 16 columns a lane and chunk in
// registers. After the sums are merged (every warp leaves its sums in the
// shared memory of all of the cluster's CTAs, one cluster barrier) the
// gradient pass walks the chunks backwards: those still in their slots are
// not read again, the others come from L2 while the rows in flight fit there
// (740 rows of 151936 bf16 do not: 863 MB read for 472 MB of rows, at half of
// HBM's rate). No wait in this kernel depends on another launch.
//
// Bound by instruction issue: 20 thread instructions an element for the
// statistic, 13 more for the gradient, at 60-70 % of the issue slots (the
// rest are the rows' serial ends and the last wave). The statistic of 8192 x
// 151936 bf16 takes 1.02 ms, where the row pass over dense bf16 rows, which
// has no codes to decode, takes 0.91. Five CTAs of 128 threads and 96
// registers an SM measured best (64 threads 1.18, 256 threads 1.20, 512
// threads 1.59 ms); the instances spill up to 80 bytes a thread at that, 16-bit
// quant rows with shifted codes most. So did two chunks at a time (one: 1.10
// ms). Clusters for many rows cost more ends than they save
// reads: the gradient of 2048 x 151936 bf16 takes 0.51 ms whole, 0.52 in
// two, 0.60 in four. A persistent kernel with a producer warp, sixteen consumer
// warps that run on from row to row and warps that merge behind them was no
// faster (statistic 1.10, gradient 0.55 ms) and is not kept.
//
// Alignment: chunks follow the 16-byte grid of the dense operand (the quant
// rows, else the gradient), so a row that starts `off` elements into a
// vector has its codes shifted by as many bytes (kOff). The first and last
// chunk, when they cross the row's ends, and chunks with masked or bad blocks
// are done apart with plain loads.
#include "kld_packed_rows.cuh"

namespace kld {
namespace {
namespace from_packed {

constexpr int kThreads = 128;
constexpr int kCtasPerSm = 5;  // 20 warps of at most 96 registers
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 2;        // chunks a warp takes at a time
constexpr int kDepth = 2;      // times kSub chunks in flight per warp
constexpr int kMaxCluster = 8;
constexpr int kMaxParts = kMaxCluster * kWarps;

struct Shared {
  Part part[kMaxParts];  // every warp of the cluster, written by its owner
  Total total;
  int ib, iq;            // lowest columns of the maxima (rank 0's are the row's)
  Token tok;
  Later later[kWarps];
  float edge[2][32];     // the last chunk's maxima, by lane
  SlowShared slow;
};

// ------------------------------------------------------------------ kernel

// grid = N * C CTAs, clusters of C = gridDim / N; slots: shared-memory slots
// per warp (>= kDepth).
template <int QT, int OT, bool kOff>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    kld_packed_rows_kernel(const Operands in, const Outputs out, int C, int slots) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared sh;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / C;
  const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t V = in.V, nb = in.nb;
  if (C > 1) cluster_arrive();  // peers may be written to once all have started
  if (tid == 0) sh.ib = sh.iq = INT_MAX;

  RowPtr rp;
  rp.bcodes = in.bcodes + r * nb * kBlock;
  rp.bheads = in.bheads + r * nb;
  rp.qheads = nullptr;
  char* grow = out.grad ? static_cast<char*>(out.grad) + r * V * Type<OT>::kBytes : nullptr;
  if (QT == kFromPack) {
    rp.quant = static_cast<const char*>(in.quant) + r * nb * kBlock;
    rp.qheads = in.qheads + r * nb;
    rp.off = kOff ? static_cast<int>((reinterpret_cast<uintptr_t>(grow) & 15u) / Type<OT>::kBytes) : 0;
  } else {
    rp.quant = static_cast<const char*>(in.quant) + r * V * Quant<QT>::kBytes;
    rp.off = kOff ? static_cast<int>((reinterpret_cast<uintptr_t>(rp.quant) & 15u) / Quant<QT>::kBytes) : 0;
  }
  const int off = kOff ? rp.off : 0;

  // This CTA's chunks [c0, c1), of which [d0, d1) lie inside the row (their
  // vectors whole, their headers and shifted codes in the row's buffers). The
  // row's first and last chunk may not; they are done apart.
  const int chunks = static_cast<int>((V + off + kChunk - 1) / kChunk);
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * rank / C);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / C);
  const int in1 = static_cast<int>((V + off) / kChunk);
  const int d0 = kOff && c0 == 0 ? 1 : c0;
  const int d1 = c1 < in1 ? c1 : in1;
  const int edge0 = c0 < c1 && c0 < d0 ? c0 : -1;
  const int edge1 = c0 < c1 && d1 < c1 && c1 - 1 != edge0 ? c1 - 1 : -1;
  // Warp w takes the pairs of chunks d0 + kSub * (w + i * kWarps), i < n.
  const int pairs = d0 < d1 ? (d1 - d0 + kSub - 1) / kSub : 0;
  const int n = warp < pairs ? (pairs - warp + kWarps - 1) / kWarps : 0;
  constexpr int kPair = kSub * Slot<QT>::kBytes;
  const LanePtr lp = lane_ptr<QT, kOff>(rp, lane);
  const uint32_t my = smem_u32(ring) + static_cast<uint32_t>(warp * slots * kPair);
  const int first = d0 + kSub * warp;
  auto load = [&](int i, int slot) {
    const int c = first + i * (kSub * kWarps);
#pragma unroll
    for (int v = 0; v < kSub; ++v)
      if (c + v < d1) fetch<QT, kOff>(lp, c + v, my + slot * kPair + v * Slot<QT>::kBytes, lane);
  };

  State st = fresh_state();
  int later = 0;  // chunks put off

  // The token's values, on their way early: needed at the very end.
  if (rank == 0 && tid == kThreads - 1) sh.tok = token_of<QT>(in, rp, r);

  // ---- sums
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    if (i < n) load(i, i);
    copy_commit();
  }
  // The row's ends, while the first copies are on their way. The last chunk's
  // maxima are kept for the end of the sums: equal ones of earlier chunks
  // come first.
  const int edge = warp == 0 ? edge0 : (warp == kWarps - 1 ? edge1 : -1);
  if (edge >= 0) {
    st = add_later<QT>(st, rp, V, edge, lane);
    if (edge == edge1) {
      sh.edge[0][lane] = st.mb;
      sh.edge[1][lane] = st.mq;
      st.mb = st.mq = neg_inf();
    }
  }
  int cur = 0, nxt = kDepth == slots ? 0 : kDepth;  // slots of chunks i and i + kDepth
  Long moved;  // sums of the chunks before the last kFold
  bool folded = false;
  for (int stop = 0, i = 0; i < n;) {
    if (i > 0) {
      st = fold(st, &moved, !folded);
      folded = true;
    }
    stop = stop + kFold / kSub < n ? stop + kFold / kSub : n;
    for (; i < stop; ++i) {
      copy_wait<kDepth - 1>();
      __syncwarp();
      int c = first + i * (kSub * kWarps);
      const int end = c + kSub < d1 ? c + kSub : d1;
      uint32_t slot = my + cur * kPair;
#pragma unroll 1
      for (; c < end; ++c, slot += Slot<QT>::kBytes) {
        float b[16], q[16];
        uint32_t qw[8];
        Heads<QT, kOff> h;
        h.load(slot + Slot<QT>::kHeads, slot + Slot<QT>::kQuant + kCodeBytes, off, lane);
        const uint32_t special = step_plain<QT, kOff>(off, slot, slot + Slot<QT>::kQuant, h, lane, b, q, qw);
        if (!add_step<QT, true>(st, b, q, qw, special, 0xffffu, c)) {
          if (later < kLater && lane == 0) sh.later[warp].chunk[later] = c;
          ++later;
        }
      }
      __syncwarp();
      if (i + kDepth < n) load(i + kDepth, nxt);
      copy_commit();
      if (++cur == slots) cur = 0;
      if (++nxt == slots) nxt = 0;
    }
  }

  // The chunks put off, `one` for each; falls: the pairs passed falling.
  auto others = [&](bool falls, auto&& one) {
    __syncwarp();
    const int listed = later < kLater ? later : kLater;
    for (int i = 0; i < listed; ++i) one(sh.later[warp].chunk[i]);
    if (later > kLater) {
      // those passed after the last one listed (a pair's chunks rise)
      const int last = sh.later[warp].chunk[kLater - 1];
      const int last_i = (last - first) / (kSub * kWarps);
      for (int i = 0; i < n; ++i) {
        for (int v = 0; v < kSub; ++v) {
          const int c = first + i * (kSub * kWarps) + v;
          const bool after = i == last_i ? c > last : (i < last_i) == falls;
          if (c < d1 && after && put_off<QT, kOff>(rp, nb, c, lane)) one(c);
        }
      }
    }
    later = 0;
    __syncwarp();
  };
  if (later > 0) {
    int since = 0;
    others(false, [&](int c) {
      if (++since == kFold) {
        st = fold(st, &moved, !folded);
        folded = true;
        since = 0;
      }
      st = add_later<QT>(st, rp, V, c, lane);
    });
  }
  if (edge >= 0 && edge == edge1) {
    if (sh.edge[0][lane] > st.mb) {
      st.mb = sh.edge[0][lane];
      st.ib = edge;
    }
    if (sh.edge[1][lane] > st.mq) {
      st.mq = sh.edge[1][lane];
      st.iq = edge;
    }
  }

  // ---- merge: lanes, then every warp of the cluster
  {
    if (folded) st = fold(st, &moved, false);
    const Part w = folded ? part_of_long(st, &moved) : part_of(st);
    if (C > 1) cluster_wait();  // every CTA of the cluster has started
    if (lane < C) {             // lane k leaves the part with CTA k
      const uint32_t* words = reinterpret_cast<const uint32_t*>(&w);
      const uint32_t at = smem_u32(&sh.part[rank * kWarps + warp]);
#pragma unroll
      for (int k = 0; k < kPartWords; ++k) {
        if (C > 1)
          store_peer(at + 4 * k, static_cast<uint32_t>(lane), words[k]);
        else
          reinterpret_cast<uint32_t*>(&sh.part[warp])[k] = words[k];
      }
    }
    __syncwarp();
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 0) merge(sh.part, C * kWarps, out.scale, grow != nullptr, &sh.total);
  __syncthreads();
  // Lowest columns of the row's maxima: the lanes that hold one look through
  // the first chunk in which it appeared; rank 0 collects.
  if (st.mb == sh.total.mb || st.mq == sh.total.mq) {
    for (int which = 0; which < 2; ++which) {
      const float m = which ? sh.total.mq : sh.total.mb;
      if ((which ? st.mq : st.mb) != m) continue;
      const int c = which ? st.iq : st.ib;
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int64_t j = static_cast<int64_t>(c) * kChunk + group_col<QT>(k / Quant<QT>::kGroup, lane) +
                          k % Quant<QT>::kGroup - off;
        x[k] = j < 0 || j >= V ? neg_inf() : (which ? quant_at<QT>(rp, j) : base_at<QT>(rp, j));
      }
      int at = INT_MAX;
      const int64_t j0 = static_cast<int64_t>(c) * kChunk - off;
#pragma unroll
      for (int k = 15; k >= 0; --k) {
        if (x[k] == m)
          at = static_cast<int>(j0 + group_col<QT>(k / Quant<QT>::kGroup, lane) + k % Quant<QT>::kGroup);
      }
      if (C > 1)
        min_peer(smem_u32(which ? &sh.iq : &sh.ib), 0u, static_cast<uint32_t>(at));
      else
        atomicMin(which ? &sh.iq : &sh.ib, at);
    }
  }
  if (!sh.total.good) {  // the same in every thread of the cluster
    copy_wait<0>();  // (the columns found above may miss what plain_scale could not hold)
    Slow s;
    slow_row<QT>(sh.slow, rp, V, s);
    if (grow) {
      if (C > 1) {  // the gradient may go over the quant rows: all have read them
        __syncwarp();
        cluster_arrive();
        cluster_wait();
      }
      const int64_t j0 = static_cast<int64_t>(c0) * kChunk - off;
      const int64_t j1 = static_cast<int64_t>(c1) * kChunk - off;
      slow_grad<QT, OT>(rp, j0 < 0 ? 0 : j0, j1 < V ? j1 : V, s, grow, out.scale);
    }
    if (C > 1) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
    __syncthreads();
    if (rank == 0 && tid == 0)
      write_row(out, sh.tok, r, s.kl, 1.0, s.mb, s.mq, log(s.Sb), log(s.Sq), s.ib, s.iq,
                    s.flags);
    return;
  }

  // ---- gradient, chunks backwards: the last `slots` of them are still here
  if (grow) {
    cur = n > 0 ? (n - 1) % slots : 0;
    char* glane = grow + (group_col<QT>(0, lane) - off) * Type<OT>::kBytes;
    const bool whole = whole_vectors<QT, OT>(glane);
    const GradScale gs(sh.total);
    for (int i = n - 1; i >= 0; --i) {
      copy_wait<kDepth - 1>();
      __syncwarp();
      int c = first + i * (kSub * kWarps);
      const int end = c + kSub < d1 ? c + kSub : d1;
      uint32_t slot = my + cur * kPair;
#pragma unroll 1
      for (; c < end; ++c, slot += Slot<QT>::kBytes) {
        float b[16], q[16];
        uint32_t qw[8];
        Heads<QT, kOff> h;
        h.load(slot + Slot<QT>::kHeads, slot + Slot<QT>::kQuant + kCodeBytes, off, lane);
        const uint32_t special = step_plain<QT, kOff>(off, slot, slot + Slot<QT>::kQuant, h, lane, b, q, qw);
        if (__any_sync(0xffffffffu, (special & 256u) != 0u)) {
          if (later < kLater && lane == 0) sh.later[warp].chunk[later] = c;
          ++later;
          continue;
        }
        if constexpr (kPacked16<QT> != 0) {
#pragma unroll
          for (int k = 0; k < 16; ++k) q[k] = q_el<kPacked16<QT>>(nullptr, qw, k);
        }
        grad_values(gs, b, q);
        char* dst = glane + static_cast<int64_t>(c) * (kChunk * Type<OT>::kBytes);
        if (whole)
          store_whole<QT, OT>(dst, b);
        else
          store_singly<QT, OT>(dst, b);
      }
      __syncwarp();
      if (i - slots >= 0) load(i - slots, cur);
      copy_commit();
      if (--cur < 0) cur = slots - 1;
    }
    if (edge >= 0) grad_later<QT, OT>(gs, rp, grow, V, edge, lane);
    if (later > 0) others(true, [&](int c) { grad_later<QT, OT>(gs, rp, grow, V, c, lane); });
  }
  copy_wait<0>();
  if (C > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  if (rank == 0 && tid == 0) {
    write_total(out, sh.tok, r, sh.total, sh.ib, sh.iq);
  }
}

// -------------------------------------------------------------------- host

// Launch shape: CTAs per row and shared-memory slots per warp.
struct Shape {
  int cluster, slots;
};
template <int QT>
Shape shape_for(int64_t N, int64_t V, int sm_count) {
  // What kCtasPerSm CTAs leave of an SM's 228 KB (1 KB a CTA is the system's).
  constexpr int most = (228 * 1024 / kCtasPerSm - static_cast<int>(sizeof(Shared)) - 1024) /
                       (kWarps * kSub * Slot<QT>::kBytes);
  static_assert(most >= kDepth, "slots");
  // What any kernel may use without an attribute of the function, which all
  // host threads would share.
  static_assert(most * kWarps * kSub * Slot<QT>::kBytes + static_cast<int>(sizeof(Shared)) <= 48 * 1024,
                "shared memory of a CTA");
  const int64_t chunks = (V + kChunk - 1) / kChunk + 1;
  // Few rows are split as long as all CTAs run at once (and a warp has more
  // than one chunk): 16 x 262144 fp32 87 us whole, 43 us in eight; 512 x 32003
  // fp32 with its gradient 91 us whole, 113 us in two.
  int c = 1;
  while (c < kMaxCluster && 2 * N * c <= static_cast<int64_t>(sm_count) * kCtasPerSm &&
         chunks > static_cast<int64_t>(c) * kWarps)
    c *= 2;
  int64_t s = (chunks + c * kWarps * kSub - 1) / (c * kWarps * kSub) + 1;
  if (s > most) s = most;
  if (s < kDepth) s = kDepth;
  return {c, static_cast<int>(s)};
}

template <int QT, int OT, bool kOff>
cudaError_t launch_shape(const Operands& in, const Outputs& out, int sm_count, cudaStream_t s) {
  const Shape sh = shape_for<QT>(in.N, in.V, sm_count);
  const int smem = kWarps * sh.slots * kSub * Slot<QT>::kBytes;
  auto kern = kld_packed_rows_kernel<QT, OT, kOff>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(in.N * sh.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(sh.cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, in, out, sh.cluster, sh.slots);
}

template <int QT, int OT>
cudaError_t launch_off(const Operands& in, const Outputs& out, int sm_count, cudaStream_t s) {
  return on_grid<QT, OT>(in, out) ? launch_shape<QT, OT, false>(in, out, sm_count, s)
            : launch_shape<QT, OT, true>(in, out, sm_count, s);
}

template <int QT>
cudaError_t launch_out(const Operands& in, const Outputs& out, kld_dtype_t ot, int sm_count,
                       cudaStream_t s) {
  switch (ot) {
    case KLD_F32: return launch_off<QT, KLD_F32>(in, out, sm_count, s);
    case KLD_BF16: return launch_off<QT, KLD_BF16>(in, out, sm_count, s);
    case KLD_F16: return launch_off<QT, KLD_F16>(in, out, sm_count, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace from_packed
}  // namespace

cudaError_t launch_packed_rows(const PackedRows& a, int sm_count, cudaStream_t stream) {
  using namespace from_packed;
  const Operands in = operands_of(a);
  const Outputs out = outputs_of(a);
  const kld_dtype_t ot = a.grad ? a.grad_dtype : KLD_F32;
  if (a.quant_codes) return launch_out<kFromPack>(in, out, ot, sm_count, stream);
  switch (a.quant_dtype) {
    case KLD_F32: return launch_out<KLD_F32>(in, out, ot, sm_count, stream);
    case KLD_BF16: return launch_out<KLD_BF16>(in, out, ot, sm_count, stream);
    case KLD_F16: return launch_out<KLD_F16>(in, out, ot, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kld
