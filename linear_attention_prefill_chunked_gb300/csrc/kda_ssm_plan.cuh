// kda_ssm_plan.cuh -- work lists of the state space scan, and the cuts of long sequences.
#pragma once

#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {

constexpr int kSsmChunk = 64;  // tokens a chunk

// Work-list entry, for every item of a sequence (or part) alike. Long sequences are cut in time where
// few items would leave SMs idle (see the planning kernel).
struct Entry {
  int32_t n, chunk0, nchunks, part;  // part: its slot of the scratch, -1: a whole sequence
  int32_t last, pad[3];              // of the sequence's parts
};
struct Split {  // a cut sequence: its parts' slots of the scratch, its slot of the states
  int32_t part0, parts;
  int64_t slot;
};
struct PlanHdr {  // over the workspace header
  uint32_t status, next_state, next_full, n_state, n_full, n_splits;
};
static_assert(sizeof(PlanHdr) <= sizeof(WsHeader), "the plan's header lies in the workspace header");

// The passes of a call follow one another on the stream, each small beside the setting up of the next: a
// pass lets the next one's blocks start as soon as its own have (grid_dep_launch_dependents), and those
// wait, before they touch global memory, until the pass is over (grid_dep_wait), and so every pass before
// it. The plan itself waits for all earlier work, and what follows the call waits for its last pass, as
// usual. (8192 tokens of 64 heads 132 -> 128 us a call, a ragged fp32 batch of 2209 tokens 58 -> 51 us.)
// after: the kernel follows one of this call's passes on the stream, and waits for it itself.
template <typename... P, typename... A>
cudaError_t launch_pass(void (*kern)(P...), dim3 grid, int block, size_t smem, bool after, cudaStream_t st,
                        const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Where the lists and the parts' scratch lie in a workspace (see the planning kernel).
struct SsmPlan {
  bool lists;          // there is room for the list of sequences
  int cap;             // most parts of cut sequences, 0: none is cut
  int items, workers;  // items a sequence, items that run at once
  int min_part;        // chunks a part has at least, or so
  PlanHdr* hdr;
  Entry *full, *state;
  Split* splits;
  float *decay, *scratch;
};
SsmPlan ssm_plan(const SsmArgs& a, int items, int workers, int min_part);
// The whole workspace a plan uses, header included (the header alone where no sequence can be cut).
size_t ssm_plan_workspace(const kda_desc_t& d, int items, int workers, int min_part);
cudaError_t launch_ssm_plan(const SsmPlan& p, const SsmArgs& a, cudaStream_t st);
cudaError_t launch_ssm_combine(const SsmPlan& p, const SsmArgs& a, cudaStream_t st);

}  // namespace kda
