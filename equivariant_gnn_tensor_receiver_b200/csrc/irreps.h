// Irreps strings ("64x0e+64x1o"), shared by the plans of all operators.
#pragma once

#include <vector>

namespace tpc {

struct Blk {
  int mul, l, p;  // multiplicity, degree, parity (+1 even, -1 odd)
};

// TPCONV_OK, TPCONV_ERR_BAD_IRREPS or TPCONV_ERR_UNSUPPORTED (degree, block count)
int parse_irreps(const char* s, std::vector<Blk>& out);

}  // namespace tpc
