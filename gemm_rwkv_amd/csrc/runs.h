// Rows 0..tokens-1 in runs of consecutive rows, a run per workgroup, the last
// one shorter.  `tokens` may be any int, so nothing is added to it.
#pragma once

namespace rq {

constexpr int run_count(int tokens, int rows) { return tokens / rows + (tokens % rows != 0); }

// One past the last row of the run that begins at `begin` < tokens.
constexpr int run_end(int tokens, int begin, int rows) { return rows < tokens - begin ? begin + rows : tokens; }

// Rows per run for `groups` runs or fewer.
constexpr int run_rows(int tokens, int groups) { return tokens ? run_count(tokens, groups) : 1; }

// The norm's rows per workgroup.  A run's first row costs the norm of the row
// before it, a long one leaves compute units idle.  Rows one, two, four, eight
// at a time, in us, at width 2048 with six mixtures and at width 2560 with one:
// 600 rows 9.7 10.8 14 22 and 7.7 7.6 9.1 13; 1025 rows 12.8 12.9 16 24 and 11
// 8.7 10 14; 2048 rows 22 18 19 27 and 20 16 14 16; 4099 rows 42 35 35 38 and 34
// 27 25 23; 16384 rows 139 134 132 153 and 117 86 77 78.  Past 4 M rows the runs
// grow, so that a grid has at most about a million workgroups.
constexpr int norm_rows(int tokens) { return tokens <= 768 ? 1 : tokens <= 1536 ? 2 : 4 + tokens / (1 << 22); }

// The head norm's rows per workgroup: a grid of at most 2^20 runs.
constexpr int gate_rows(int tokens) { return 1 + tokens / (1 << 20); }

}  // namespace rq
