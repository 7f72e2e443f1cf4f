// kv_status.h -- the spread status of the paged-cache calls, for the status
// readers.
#pragma once

namespace dspark {

// Words of the head of a spread status, and the first CTA's word.
constexpr int kSpreadHeadWords = 4;
constexpr int kMaxStatusCtas = 2044;

// Whether a workspace's first words are the head of a status that is spread
// over one word a CTA (kv_common.cuh), and over how many.
bool spread_status(const unsigned* head, unsigned* count);

}  // namespace dspark
