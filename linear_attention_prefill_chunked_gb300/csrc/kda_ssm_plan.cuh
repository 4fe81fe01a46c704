// kda_ssm_plan.cuh -- work lists of the state space scan, and the cuts of long sequences.
#pragma once

#include "kda_internal.cuh"

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
// The whole workspace a plan uses, header included.
size_t ssm_plan_workspace(const kda_desc_t& d, int items, int workers);
cudaError_t launch_ssm_plan(const SsmPlan& p, const SsmArgs& a, cudaStream_t st);
cudaError_t launch_ssm_combine(const SsmPlan& p, const SsmArgs& a, cudaStream_t st);
// SMs of the current device (152, for sizes asked for where there is none).
int gpu_sms();

}  // namespace kda
