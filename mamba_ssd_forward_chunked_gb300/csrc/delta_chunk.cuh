// The chunked form of the gated delta rule (delta_chunk.cu), for whole prompts.
#pragma once
#include "delta.cuh"

namespace ssd {

// The chunks of a pair of launches.
struct DeltaChunks {
  int first, count, last;  // chunks of 64 tokens from `first` on; last: the sequences end with them
  int vectors;             // x, Bm, Cm and y are rows of 16-byte vectors
  int follows;             // a pair of the same call came before, in the other buffer
  uint8_t* records;        // [batch][nheads][count]: what the first launch leaves for the second
  uint8_t* rows;           // [batch][ngroups][count]: and K and Q of the group
  float* carry;            // [batch][nheads][headdim][dstate]: states between pairs of launches
  uint64_t limit_ns;       // of a wait
};

// Whether these sizes take the chunked form.
bool delta_chunked(int dtype, int64_t seqlen, int dstate);
// Bytes of its workspace.
size_t delta_chunks_workspace(const DeltaParams& p);
ssd_status launch_delta_chunks(const DeltaParams& p, void* workspace, cudaStream_t stream);

}  // namespace ssd
