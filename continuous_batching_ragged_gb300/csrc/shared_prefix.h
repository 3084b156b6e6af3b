// What the kernels of a step with shared prefixes hand to one another: the plan
// writes it, in the caller's workspace.
#pragma once

#include "kernels.h"

namespace cb {

// A piece of the prefix phase: the query rows of one row tile or two, of one
// key/value head, over one KV segment of their group's prefix.
struct alignas(16) Piece {
  int s0;                      // the group's first sequence: its table holds the prefix's blocks
  int tok0, ntok;              // query tokens
  int hk;                      // key/value head
  int j0, nt;                  // KV tiles
  int shared;                  // keys of the prefix
  int rec;                     // this piece's (first) record of each row
  int alt;                     // 1: one row tile, KV tiles alternate over the two slots
  int pad[3];
};
static_assert(sizeof(Piece) == 48, "piece");

// One row tile of a sequence over one chunk of its own keys, for every key/value head.
struct alignas(16) SuffixItem {
  int s;
  int tok0, q_len;             // the sequence's packed rows
  int row0;                    // first row of the tile (row = token * G + head of the group)
  int k0, k1;                  // own keys of the chunk (0 = the first key behind the prefix)
  int ctx;                     // own keys of the sequence
  int skip;                    // blocks of the table that the prefix covers
  int base;                    // the sequence's first own record
  int nch, chunk;              // chunks of the sequence, this one
  int direct;                  // 1: nothing to join, the rows are written to out
};
static_assert(sizeof(SuffixItem) == 48, "item");

struct PrefixWork {
  const int32_t* cu_groups;    // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  const int32_t* context_lens; // [num_seqs], whole
  int32_t num_groups;
  int32_t num_sms;
  int32_t tile_tokens;         // query tokens per row tile of the prefix kernel
  int32_t max_warp_rows;       // sequences with more query rows per key/value head are prefill chunks
  int32_t suffix_units;        // warps' units that the chunk length aims for
  int32_t piece_cap, item_cap;
  int64_t rec_cap, own_cap;
  uint32_t tag;
  // in the workspace
  int32_t* header;             // [0] pieces, [1] prefix records per row (stride), [2] call tag, [3] piece
                               // claims, [4] suffix items, [5] suffix claims
  int32_t* suffix_lens;        // [num_seqs] keys behind the prefix (0: left out)
  int4* seq_info;              // [num_seqs] see PrefixView
  int4* groups;                // [num_groups] (first sequence, first token, tokens, shared keys)
  int32_t* first_piece;        // [num_groups + 1]
  Piece* pieces;
  SuffixItem* items;
  int4* token_info;            // [num_tokens] (prefix records, first own record of head 0, own records per head, -)
  float* recs;                 // prefix records [token][query head][stride]
  float* own_recs;
};

constexpr int kSuffixWarps = 8;          // warps of a suffix CTA, each with units of its own

// The rows' own keys (sequences that are not prefill chunks), then the join of
// every row that has more than one record.
cb_status launch_suffix(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream);
cb_status launch_join(const AttnArgs& a, const PrefixWork& w, cudaStream_t stream);

}  // namespace cb
