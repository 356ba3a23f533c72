// The attention kernel of spec_attend_rows.cu over what a row does not share with its group (spec_attend_shared).
#define SPEC_ATTEND_PART kOwn
#include "spec_attend_rows.cu"
